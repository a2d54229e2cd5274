"""Host-side pieces of bench.py, without a GPU: the clock sampler (against a stand-in NVML
module that only answers reads) and the comment-insensitive code digest that pins the
committed ncu traffic numbers to the kernel code they were captured on."""
import importlib.util
import os
import time

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def bench():
    spec = importlib.util.spec_from_file_location("bench_under_test", os.path.join(ROOT, "bench.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


class FakeNVML:
    """Answers the read calls the sampler makes; records that nothing else is called."""
    NVML_CLOCK_SM = 1

    def __init__(self, clocks, reasons, fail_init=False):
        self.clocks, self.reasons, self.fail_init = list(clocks), reasons, fail_init
        self.calls = []

    def nvmlInit(self):
        self.calls.append("init")
        if self.fail_init:
            raise RuntimeError("no driver")

    def nvmlDeviceGetHandleByUUID(self, uuid):
        self.calls.append("uuid")
        return "h"

    def nvmlDeviceGetHandleByIndex(self, i):
        self.calls.append("index")
        return "h"

    def nvmlDeviceGetMaxClockInfo(self, h, kind):
        assert kind == self.NVML_CLOCK_SM
        return 1965

    def nvmlDeviceGetClockInfo(self, h, kind):
        assert kind == self.NVML_CLOCK_SM
        self.calls.append("clk")
        return self.clocks[self.calls.count("clk") % len(self.clocks)]

    def nvmlDeviceGetCurrentClocksEventReasons(self, h):
        return self.reasons


def test_clock_sampler_reads_nvml_and_maps_reason_bits(bench):
    nv = FakeNVML([1965, 1965, 1950], reasons=0x4 | 0x1)   # sw power cap (+ idle bit, not reported)
    with bench.ClockSampler(0, nvml=nv, use_smi=False) as clk:
        time.sleep(0.06)
    s = clk.summary()
    assert s["samples"] >= 3
    assert s["sm_max_mhz"] == 1965.0
    assert 1950 <= s["sm_mhz"] <= 1965
    assert s["reasons"] == ["sw_power_cap"]
    assert set(nv.calls) <= {"init", "uuid", "index", "clk"}


def test_clock_sampler_reports_throttling_reasons(bench):
    nv = FakeNVML([1200], reasons=0x8 | 0x40)
    with bench.ClockSampler(0, nvml=nv, use_smi=False) as clk:
        time.sleep(0.03)
    s = clk.summary()
    assert s["reasons"] == ["hw_slowdown", "hw_thermal_slowdown"]
    assert s["sm_mhz"] == 1200.0


def test_clock_sampler_without_nvml_says_so(bench):
    nv = FakeNVML([1965], reasons=0, fail_init=True)
    with bench.ClockSampler(0, nvml=nv, use_smi=False) as clk:
        pass
    s = clk.summary()
    assert s["sm_mhz"] is None and s["reasons"]


def test_code_digest_ignores_comments_and_layout_but_not_code(bench, tmp_path):
    a = tmp_path / "a.cuh"
    b = tmp_path / "b.cuh"
    c = tmp_path / "c.cuh"
    a.write_text('int f(int x) { return x + 1; }  // one\nconst char *s = "a // b";\n')
    b.write_text('/* header */\nint f(int x)\n{\n  return x + 1;   // one more comment\n}\nconst char *s = "a // b";\n')
    c.write_text('int f(int x) { return x + 2; }\nconst char *s = "a // b";\n')
    assert bench.code_digest(str(a)) == bench.code_digest(str(b))
    assert bench.code_digest(str(a)) != bench.code_digest(str(c))



@pytest.mark.parametrize("workload", ["decode_b1_l40", "prefill_t4096_l40"])
def test_traffic_pins_hold(bench, workload):
    """The committed ncu traffic belongs to the kernels as they are: their code is the code captured."""
    nbytes, how = bench.kernel_traffic(workload)
    assert nbytes is not None, how


RANGE = "one-launch decode: an activation beyond the fp16 operand range (|v| >= 65520); e0_debug_force_general ..."


@pytest.mark.parametrize("chained,code,msg,excused", [
    (True, -7, RANGE, True), (False, -7, RANGE, False), (True, -7, "routing rejected on the device", False),
    (True, -6, "a bounded device wait gave up", False), (True, -2, "launch k_decode: out of memory", False), (True, -1, RANGE, False)])
def test_a_decode_variant_excuses_the_fp16_range_alone(bench, chained, code, msg, excused):
    import int4_expert_streaming_prerouter_b200 as e0
    modes = []

    def steps_in(mode):
        modes.append(mode)
        if mode != 2:
            raise e0.E0Error(code, msg)
        return 1.0, {}, 7
    if not excused:
        with pytest.raises(e0.E0Error):
            bench._timed_variant(steps_in, 0, chained)
        assert modes == [0]
        return
    timed, mode, kernel = bench._timed_variant(steps_in, 0, chained)
    assert timed == (1.0, {}, 7) and mode == 2 and modes == [0, 2] and "fp16 operand range" in kernel


def test_a_decode_variant_without_an_error_is_the_one_asked_for(bench):
    timed, mode, kernel = bench._timed_variant(lambda mode: (2.0, {}, mode), 1, False)
    assert timed == (2.0, {}, 1) and mode == 1 and "k_decode" in kernel


def test_the_library_says_what_is_excused():
    """The words that the excuse looks for are the library's own."""
    src = open(os.path.join(ROOT, "int4_expert_streaming_prerouter_b200", "csrc", "e0_api.cu"), encoding="utf-8").read()
    at = src.index("err & kDerrRange")
    assert "E0_ERR_DEVICE" in src[at:at + 200] and "fp16 operand range" in src[at:at + 200]
