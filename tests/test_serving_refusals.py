"""The operators around the attention (add_rmsnorm, int4_linear, moe_layer_few) refuse what
they do not take before anything is enqueued.  CPU only: the addresses are never read."""
import ctypes

import pytest
import torch

import int4_expert_streaming_prerouter_b200 as e0

P = 1 << 20          # an aligned address that no call reads


def norm(**kw):
    a = dict(h=P, h_stride=256, delta=None, delta_f32=0, delta_stride=0, norm_w=P, eps=1e-6, T=2, d=256, h_out=None,
             h_out_stride=0, x=P, x_stride=256, q8=None, q8_format=0, q8_stride=0, q8_group=0, q8_scale=None, stream=None)
    assert set(kw) <= set(a)
    return e0.lib().e0_add_rmsnorm(*(a | kw).values())


@pytest.mark.parametrize("bad", [
    dict(h=None), dict(T=-1), dict(d=0), dict(d=32769, h_stride=40000, x_stride=40000), dict(x=None), dict(norm_w=None),
    dict(h_stride=255), dict(x_stride=255), dict(delta=P, delta_stride=255), dict(delta=P, delta_stride=256, delta_f32=2),
    dict(h_out=P, h_out_stride=0), dict(q8=P, q8_stride=256, q8_format=1),                      # no scales
    dict(q8=P, q8_stride=256, q8_format=0, q8_scale=P), dict(q8=P, q8_stride=256, q8_format=3, q8_scale=P),
    dict(q8=P, q8_stride=256, q8_format=1, q8_scale=P, q8_group=32), dict(q8=P, q8_stride=9, q8_format=1, q8_scale=P),
])
def test_add_rmsnorm_refuses(bad):
    assert norm(**bad) == -1
    assert b"add_rmsnorm" in e0.lib().e0_last_error()


def test_add_rmsnorm_of_no_rows_is_nothing():
    assert norm(T=0) == 0


def linear(mat=None, **kw):
    m = dict(codes=P, scale=P, min=P, n=48, k=256, group=64, lora_A=None, lora_B=None, lora_rank=0, lora_scale=1.0)
    assert set(mat or {}) <= set(m)
    m = e0.Int4Mat(*(m | (mat or {})).values())
    a = dict(x=P, x_format=0, x_stride=256, x_scale=None, x_group=0, T=2, y=P, y_f32=0, y_stride=48, stream=None)
    assert set(kw) <= set(a)
    return e0.lib().e0_int4_linear(ctypes.byref(m), *(a | kw).values())


@pytest.mark.parametrize("mat,bad", [
    (dict(codes=None), {}), (dict(scale=None), {}), (dict(min=None), {}), (dict(n=0), {}), (dict(k=0), {}),
    (dict(group=32), {}), (dict(k=192, group=128), {}), (dict(k=224), {}), (dict(codes=P + 8), {}),
    (dict(lora_A=P), {}), (dict(lora_B=P, lora_rank=4), {}), (dict(lora_A=P, lora_B=P, lora_rank=33), {}),
    (dict(lora_A=P, lora_B=P, lora_rank=0), {}), (dict(lora_A=P + 2, lora_B=P, lora_rank=4), {}),
    ({}, dict(x=None)), ({}, dict(y=None)), ({}, dict(T=-1)), ({}, dict(x_format=3)), ({}, dict(x_format=-1)),
    ({}, dict(x_scale=P)), ({}, dict(x_format=1)), ({}, dict(x_format=1, x_scale=P, x_group=32)),
    (dict(k=192), dict(x_format=1, x_scale=P, x_group=128)), ({}, dict(x=P + 8)), ({}, dict(x_stride=255)),
    ({}, dict(x_stride=260)), ({}, dict(y_stride=47)), ({}, dict(y_f32=2)), ({}, dict(T=524281)),
])
def test_int4_linear_refuses(mat, bad):
    assert linear(mat, **bad) == -1
    assert b"int4_linear" in e0.lib().e0_last_error()


def test_int4_linear_of_no_tokens_is_nothing():
    assert linear(T=0) == 0


def few(dims=None, layer=None, **kw):
    D = e0.make_dims(*(dims or (256, 16, 128, 4, 8)))
    L = dict(experts=P, shared=P, lora_Ag=None, lora_Bg=None, lora_Au=None, lora_Bu=None, lora_Ad=None, lora_Bd=None,
             router_w=P, norm_w=P)
    assert set(layer or {}) <= set(L)
    L = e0.Layer(*(L | (layer or {})).values())
    a = dict(h=P, delta=None, T=2, route_idx=None, h_out=None, y=P, y_f32=None, idx=None, gates=None, workspace=P,
             workspace_bytes=1 << 30, dev_status=None, stream=None)
    assert set(kw) <= set(a)
    return e0.lib().e0_moe_layer_few(ctypes.byref(D), ctypes.byref(L), *(a | kw).values())


@pytest.mark.parametrize("dims,layer,bad", [
    (None, None, dict(h=None)), (None, None, dict(y=None)), (None, None, dict(T=0)), (None, None, dict(T=65)),
    (None, None, dict(T=-1)), (None, None, dict(workspace=None)), (None, None, dict(workspace=P + 16)),
    (None, None, dict(workspace_bytes=100)), (None, None, dict(h=P + 2)), (None, None, dict(delta=P + 2)),
    (None, None, dict(h_out=P + 2)), (None, dict(experts=None), {}), (None, dict(shared=None), {}),
    (None, dict(router_w=None), {}), (None, dict(norm_w=None), {}), (None, dict(experts=P + 8), {}),
    (None, dict(lora_Ag=P), {}), (None, dict(lora_Bd=P), {}), ((100, 16, 128, 4, 8), None, {}),
    ((256, 257, 128, 4, 8), None, {}), ((256, 16, 100, 4, 8), None, {}), ((256, 16, 128, 9, 8), None, {}),
    ((256, 3, 128, 4, 8), None, {}), ((256, 16, 128, 4, 33), None, {}), ((8192, 16, 128, 4, 8), None, {}),
])
def test_moe_layer_few_refuses(dims, layer, bad):
    assert few(dims, layer, **bad) == -1
    assert b"moe_layer_few" in e0.lib().e0_last_error()


def test_moe_layer_few_workspace_size():
    D, n, last = e0.make_dims(2048, 256, 512, 4, 16), ctypes.c_size_t(0), 0
    for T in (1, 2, 8, 64):
        assert e0.lib().e0_moe_layer_few_workspace(ctypes.byref(D), T, ctypes.byref(n)) == 0
        # x, logits, LoRA intermediates and a of T tokens at least; no more with fewer tokens
        assert n.value >= T * (2 * 2048 + 4 * 256 + 8 * 16 + 2 * 5 * 512) and n.value >= last
        last = n.value
    for T in (0, 65):
        assert e0.lib().e0_moe_layer_few_workspace(ctypes.byref(D), T, ctypes.byref(n)) == -1


def test_the_binding_refuses_what_does_not_fit():
    bf16 = torch.bfloat16
    h, w = torch.zeros(2, 64, dtype=bf16), torch.zeros(64, dtype=bf16)
    with pytest.raises(ValueError):                       # not on a GPU
        e0.add_rmsnorm(h, w, x=torch.zeros_like(h))
    with pytest.raises(TypeError):
        e0.add_rmsnorm(h.float(), w, x=torch.zeros_like(h))
    with pytest.raises(ValueError):
        e0.add_rmsnorm(h, w, delta=torch.zeros(2, 32, dtype=bf16), x=h)
    with pytest.raises(ValueError):
        e0.add_rmsnorm(h, w[:32], x=torch.zeros_like(h))
    with pytest.raises(TypeError):
        e0.add_rmsnorm(h, w, q8=torch.zeros(2, 64, dtype=torch.uint8))
    with pytest.raises(ValueError):
        e0.add_rmsnorm(h, w, q8=torch.zeros(2, 64, dtype=torch.int8), q8_group=32)
    with pytest.raises(ValueError):                       # transposed: a row's channels are apart
        e0.add_rmsnorm(torch.zeros(64, 2, dtype=bf16).T, w, x=h)
    codes, s = torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 2, dtype=bf16)
    with pytest.raises(ValueError):
        e0.Int4Linear(codes, torch.zeros(8, 3, dtype=bf16), torch.zeros(8, 3, dtype=bf16))
    with pytest.raises(ValueError):
        e0.Int4Linear(codes, s, s[:4])
    with pytest.raises(ValueError):
        e0.Int4Linear(codes, s, s, lora_A=torch.zeros(4, 128, dtype=bf16))
    lin = e0.Int4Linear(codes, s, s)
    assert (lin.n, lin.k, lin.group) == (8, 128, 64)
    with pytest.raises(TypeError):
        lin(torch.zeros(1, 128))
    with pytest.raises(ValueError):
        lin(torch.zeros(1, 64, dtype=bf16), y=torch.zeros(1, 8, dtype=bf16))
    with pytest.raises(ValueError):
        lin(torch.zeros(1, 128, dtype=torch.int8), x_scale=torch.zeros(1, 3), y=torch.zeros(1, 8, dtype=bf16))
    ml = e0.MoeLayer(e0.make_dims(256, 16, 128, 4, 8), {"router_w": torch.zeros(16, 256, dtype=bf16)})
    with pytest.raises(ValueError):
        ml.few(torch.zeros(1, 128, dtype=bf16), y=torch.zeros(1, 256, dtype=bf16), workspace=codes)
    with pytest.raises(e0.E0Error):
        ml.few_workspace(65)


@pytest.mark.parametrize("call,bad", [
    (norm, dict(h=P + 1)), (norm, dict(norm_w=P + 1)), (norm, dict(x=P + 1)), (norm, dict(h_out=P + 1, h_out_stride=256)),
    (norm, dict(delta=P + 1, delta_stride=256)), (norm, dict(delta=P + 2, delta_stride=256, delta_f32=1)),
    (norm, dict(q8=P, q8_stride=256, q8_format=1, q8_scale=P + 2)),
    (linear, dict(mat=dict(scale=P + 1))), (linear, dict(mat=dict(min=P + 1))),
    (linear, dict(mat=dict(lora_A=P, lora_B=P + 1, lora_rank=4))), (linear, dict(x_format=1, x_scale=P + 2)),
    (linear, dict(y=P + 1)), (linear, dict(y=P + 2, y_f32=1)),
    (few, dict(y=P + 1)), (few, dict(y_f32=P + 2)), (few, dict(route_idx=P + 2)), (few, dict(idx=P + 2)), (few, dict(gates=P + 2)),
    (few, dict(dev_status=P + 2)),
    (few, dict(layer=dict(lora_Ag=P, lora_Bg=P + 1, lora_Au=P, lora_Bu=P, lora_Ad=P, lora_Bd=P))),
    (few, dict(layer=dict(lora_Ag=P, lora_Bg=P, lora_Au=P, lora_Bu=P + 1, lora_Ad=P, lora_Bd=P))),
    (few, dict(layer=dict(lora_Ag=P, lora_Bg=P, lora_Au=P, lora_Bu=P, lora_Ad=P, lora_Bd=P + 1))),
])
def test_addresses_between_elements_are_refused(call, bad):
    """An address that is no multiple of its element's size would be a misaligned access on the device."""
    assert call(**bad) == -1
    assert b"aligned" in e0.lib().e0_last_error()


class FakeLibrary:
    """Answers the calls of a context's life without a GPU; records that nothing is launched."""

    def __init__(self):
        self.launched = 0

    def e0_create(self, dims, n, tokens, out):
        out._obj.value = 1
        return 0

    def e0_register_model(self, ctx, layers, heads):
        return 0

    def e0_destroy(self, ctx):
        return 0

    def e0_last_error(self):
        return b""

    def e0_moe_layer_few(self, *args):
        self.launched += 1
        return 0

    def e0_moe_layer_few_workspace(self, dims, T, n):
        n._obj.value = 64
        return 0


def few_layer(d=256, E=16, I=128, r=8, device="cpu"):
    bf16 = dict(dtype=torch.bfloat16, device=device)
    blob = 3 * (I * d // 2 + 4 * I * (d // 64))
    return {"experts": torch.zeros((E, blob), dtype=torch.uint8, device=device),
            "shared": torch.zeros(blob, dtype=torch.uint8, device=device),
            "router_w": torch.zeros((E, d), **bf16), "norm_w": torch.zeros(d, **bf16),
            "lora_Ag": torch.zeros((r, d), **bf16), "lora_Bg": torch.zeros((I, r), **bf16),
            "lora_Au": torch.zeros((r, d), **bf16), "lora_Bu": torch.zeros((I, r), **bf16),
            "lora_Ad": torch.zeros((r, I), **bf16), "lora_Bd": torch.zeros((d, r), **bf16)}


def test_a_closed_context_runs_no_layer(monkeypatch):
    """close() lets go of the weights; a call after it would read freed memory."""
    fake = FakeLibrary()
    monkeypatch.setattr(e0, "lib", lambda: fake)
    monkeypatch.setattr(e0, "_call", lambda X, dev, stream, fn, *args: fake.e0_moe_layer_few(*args))
    monkeypatch.setattr(e0, "_torch_names", None)
    monkeypatch.setattr(FakeLibrary, "e0_add_rmsnorm", None, raising=False)
    monkeypatch.setattr(FakeLibrary, "e0_int4_linear", None, raising=False)
    ctx = e0.Context(256, 16, 128, 4, 8, 1, 8)
    ctx.register_model([few_layer()])
    h = torch.zeros((1, 256), dtype=torch.bfloat16)
    ctx.moe_layer_few(0, h)
    assert fake.launched == 1
    ctx.close()
    with pytest.raises(e0.E0Error):
        ctx.moe_layer_few(0, h)
    assert fake.launched == 1


def few_handles(monkeypatch, layer, dims=(256, 16, 128, 4, 8)):
    """The two ways to a layer: a call of one token that MoeLayer and one that a context makes, counted by the library."""
    fake = FakeLibrary()
    monkeypatch.setattr(e0, "lib", lambda: fake)
    monkeypatch.setattr(e0, "_call", lambda X, dev, stream, fn, *args: fake.e0_moe_layer_few(*args))
    monkeypatch.setattr(e0, "_torch_names", None)
    monkeypatch.setattr(FakeLibrary, "e0_add_rmsnorm", None, raising=False)
    monkeypatch.setattr(FakeLibrary, "e0_int4_linear", None, raising=False)
    h = torch.zeros((1, dims[0]), dtype=torch.bfloat16)

    def by_handle():
        e0.MoeLayer(e0.make_dims(*dims), layer).few(h)

    def by_context():
        ctx = e0.Context(*dims, 1, 8)
        ctx.register_model([layer])
        ctx.moe_layer_few(0, h)
    return fake, (by_handle, by_context)


@pytest.mark.parametrize("change", [
    dict(experts=lambda t: t[:15]), dict(experts=lambda t: t[:, :-64].contiguous()), dict(experts=lambda t: t.view(torch.int8)),
    dict(shared=lambda t: t[:-2]), dict(shared=lambda t: t[None]), dict(router_w=lambda t: t.float()),
    dict(router_w=lambda t: t[:, :128].contiguous()), dict(router_w=lambda t: t.half()), dict(norm_w=lambda t: t[:255]),
    dict(norm_w=lambda t: t.view(torch.int16)), dict(lora_Ag=lambda t: t[:7]), dict(lora_Bg=lambda t: t[:, :4].contiguous()),
    dict(lora_Au=lambda t: t.T.contiguous()), dict(lora_Bu=lambda t: t[:64]), dict(lora_Ad=lambda t: t.repeat(2, 1)),
    dict(lora_Bd=lambda t: t.float()), dict(router_w=lambda t: t.to("meta")), dict(experts=lambda t: t.T),
])
def test_moe_layer_weights_that_do_not_fit_the_dims(change, monkeypatch):
    """Tensors of another shape or type, or on another device, would be read past their ends, or as what they are not."""
    (name, make), = change.items()
    layer = few_layer()
    layer[name] = make(layer[name])
    fake, calls = few_handles(monkeypatch, layer)
    for call in calls:
        with pytest.raises((ValueError, TypeError)):
            call()
    assert fake.launched == 0


def test_moe_layer_weights_that_fit(monkeypatch):
    plain = few_layer()
    no_lora = {n: t for n, t in plain.items() if not n.startswith("lora_")}
    for layer, dims in ((plain, (256, 16, 128, 4, 8)), (no_lora, (256, 16, 128, 4, 8)), (no_lora, (256, 16, 128, 4, 0)),
                        (few_layer(r=3), (256, 16, 128, 4, 3)), (plain | {"lora_Ag": None, "lora_Bg": None}, (256, 16, 128, 4, 8))):
        fake, calls = few_handles(monkeypatch, layer, dims)
        for call in calls:
            call()
        assert fake.launched == 2


def test_moe_layer_on_another_device_than_its_input(monkeypatch):
    fake, _ = few_handles(monkeypatch, few_layer())
    ml = e0.MoeLayer(e0.make_dims(256, 16, 128, 4, 8), few_layer())
    h = torch.zeros((1, 256), dtype=torch.bfloat16)
    ml.few(h)
    ml._dev = 1                                          # as weights of the second GPU have it
    with pytest.raises(ValueError):
        ml.few(h)
    assert fake.launched == 1
