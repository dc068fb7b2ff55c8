"""Where the buffers of weights and optimiser groups are, and how long they
live: checks of the binding that need no GPU (tensors that say they are on one
stand in for its tensors, and no library call is made)."""
import contextlib
import ctypes
import gc
import types
import weakref

import pytest
import torch


recorded = {}  # buffers by the stream that their memory waits for


class Cuda(torch.Tensor):
    """A host tensor that says it is on CUDA device `index`."""
    index = 0

    def get_device(self):
        return self.index

    def record_stream(self, stream):
        recorded.setdefault(stream, set()).add(self.data_ptr())


def cuda(t, index=0):
    t = t.as_subclass(Cuda)
    t.index = index
    return t


@pytest.fixture()
def L(monkeypatch):
    """The binding with device 0 as the current one; `called` lists the library functions that were reached."""
    from layer_streamed_qlora_b200 import _lib
    called = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: called.append(name) or 0

    monkeypatch.setattr(_lib, "lib", lambda: Library())
    monkeypatch.setattr(_lib, "_stream", lambda stream=None: None)
    monkeypatch.setattr(_lib, "_raw_stream", lambda stream, dev: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    ns = types.SimpleNamespace(**{k: getattr(_lib, k) for k in dir(_lib) if not k.startswith("__")})
    ns.called, ns.module = called, _lib
    return ns


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def weights(L, on):
    """One weight [64, 128] of each storage with its buffers made by `on`."""
    return [L.weight_mxfp4(on(u8(64, 64)), on(u8(64, 16)), 64, 128),
            L.weight_nf4(on(u8(64, 64)), on(torch.zeros(64, 2)), 64, 128),
            L.weight_bf16(on(torch.zeros(64, 128, dtype=torch.bfloat16)))]


def calls(L, W):
    b = lambda *s: cuda(torch.zeros(*s, dtype=torch.bfloat16))
    A, B, x, y, u = b(8, 128), b(64, 8), b(4, 128), b(4, 64), b(8, 8)
    ws = cuda(u8(256))
    layer = L.LayerWeights(W, W, W, W, None, None)
    cfg = L.LayerCfg()
    return [lambda: L.soup_linear_fwd(W, x, y), lambda: L.soup_linear_bwd(W, y, x),
            lambda: L.soup_lora_linear_fwd(W, A, B, 8, 1.0, x, 4, y, u),
            lambda: L.soup_lora_linear_bwd(W, A, B, 8, 1.0, x, u, y, 4, x, A, B, ws),
            lambda: L.soup_lora_linear_bwd_noalloc(W, A, B, 8, 1.0, x, u, y, 4, x, A, B),
            lambda: L.soup_decoder_layer_fwd(layer, None, cfg, x, 1, 4, x, False, ws),
            lambda: L.soup_decoder_layer_bwd(layer, None, cfg, x, x, 1, 4, x, None, False, ws),
            lambda: L.soup_decoder_layer_fwd_keep(layer, None, cfg, x, 1, 4, x, False, ws, ws),
            lambda: L.soup_decoder_layer_bwd_kept(layer, None, cfg, x, x, 1, 4, x, None, False, ws, ws),
            lambda: L.soup_decoder_layer_fwd_save(layer, None, cfg, x, 1, 4, x, False, ws, ws),
            lambda: L.soup_decoder_layer_bwd_saved(layer, None, cfg, x, x, 1, 4, x, None, False, ws, ws)]


@pytest.mark.parametrize("kind", range(3))
def test_weights_in_host_memory_or_on_another_device_are_refused(L, kind):
    for on, where in ((lambda t: t, "host memory"), (lambda t: cuda(t, 1), "on device 1")):
        for call in calls(L, weights(L, on)[kind]):
            with pytest.raises(ValueError, match=where):
                call()
    assert not L.called


@pytest.mark.parametrize("kind", range(3))
def test_weights_on_the_current_device_and_bare_addresses_are_taken(L, kind):
    W = weights(L, cuda)[kind]
    bare = L.SoupWeight()
    ctypes.memmove(ctypes.byref(bare), ctypes.byref(W), ctypes.sizeof(W))
    for w in (W, bare):
        todo = calls(L, w)
        for call in todo:
            call()
        assert len(L.called) == len(todo)
        L.called.clear()


def test_buffers_of_one_weight_or_layer_on_two_devices_are_refused(L):
    with pytest.raises(ValueError, match="different devices"):
        L.weight_mxfp4(cuda(u8(64, 64)), u8(64, 16), 64, 128)
    with pytest.raises(ValueError, match="different devices"):
        L.weight_nf4(cuda(u8(64, 64)), cuda(torch.zeros(64, 2), 1), 64, 128)
    a, b = weights(L, cuda)[0], weights(L, lambda t: cuda(t, 1))[0]
    with pytest.raises(ValueError, match="different devices"):
        L.LayerWeights(a, a, b, a, None, None)


@pytest.mark.parametrize("kind", range(3))
@pytest.mark.parametrize("layer", [False, True])
def test_weights_and_layers_keep_their_buffers(L, kind, layer):
    """Buffers that only the weight was made from live as long as it, or the layer, does."""
    made = []

    def on(t):
        made.append(weakref.ref(t.untyped_storage()))
        return t

    W = weights(L, on)
    made = made[:2] if kind == 0 else made[2:4] if kind == 1 else made[4:]
    keep = L.LayerWeights(W[kind], W[kind], W[kind], W[kind], None, None) if layer else W[kind]
    del W
    gc.collect()
    assert all(r() is not None for r in made)
    del keep
    gc.collect()
    assert not any(r() is not None for r in made)


def adamw_group(L, monkeypatch, **kw):
    """A group of two tensors, the second without a bf16 copy, and the addresses of its buffers."""
    recorded.clear()
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: cuda(empty(*a, **k)))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    f = lambda: cuda(torch.zeros(64))
    parts = [dict(theta=f(), theta_bf16=cuda(torch.zeros(64, dtype=torch.bfloat16)), grad=f(), m=f(), v=f()),
             dict(theta=f(), theta_bf16=None, grad=f(), m=f(), v=f(), name="second")]
    group = L.AdamWGroup(parts, 32, **kw)
    buffers = {t.data_ptr() for p in parts for t in p.values() if isinstance(t, torch.Tensor)}
    return group, buffers | {group._tables.data_ptr()}


HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, grad_scale=1.0, t=1)


def test_a_group_that_goes_leaves_its_memory_to_the_streams_it_stepped_on(L, monkeypatch):
    """The memory of the tables, and of tensors that nothing else holds, must not be handed out before steps on
    other streams have read it."""
    side = type("Side", (), {"cuda_stream": 77})()
    now = type("Now", (), {"cuda_stream": 5})()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now)
    monkeypatch.setattr(L.module, "_raw_stream", lambda stream, dev: 5 if stream is None else stream.cuda_stream)
    group, buffers = adamw_group(L, monkeypatch)
    for stream in (side, None, side, None):
        group.step(**HP, stream=stream)
    assert L.called.count("soup_adamw_group_step") == 4 and not recorded
    del group
    gc.collect()
    assert recorded == {side: buffers, now: buffers}


def test_a_group_that_never_stepped_or_failed_goes_quietly(L, monkeypatch):
    group, _ = adamw_group(L, monkeypatch)
    del group
    with pytest.raises(ValueError, match="no tensors"):
        L.AdamWGroup([])
    gc.collect()
    assert not recorded
