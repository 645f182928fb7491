"""Every tensor of a call lies on the device of its queries, checked before the call (CPU, with
tensors that say which GPU they are on)."""
import inspect

import pytest
import torch

import ring_collectives_gb300 as rc

P, T, HQ, HKV, D = 2, 6, 4, 2, 64


class On(torch.Tensor):
    """A host tensor that claims to be on GPU `gpu`; its memory is never followed."""
    gpu = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.gpu


def on(gpu, *shape, dtype=torch.bfloat16):
    t = torch.zeros(shape, dtype=dtype).as_subclass(On)
    t.gpu = gpu
    return t


def attention(backward):
    f32, i32 = torch.float32, torch.int32
    a = dict(q=on(1, P, T, HQ, D), k=on(1, P, T, HKV, D), v=on(1, P, T, HKV, D), out=on(1, P, T, HQ, D),
             lse=on(1, P, T, HQ, dtype=f32))
    if backward:
        a |= dict(dout=on(1, P, T, HQ, D), dq=on(1, P, T, HQ, D), dk=on(1, P, T, HKV, D), dv=on(1, P, T, HKV, D))
    return a | dict(cu_q=on(1, 3, dtype=i32), cu_k=on(1, 3, dtype=i32), used_k=on(1, 2, dtype=i32),
                    workspace=on(1, 4096, dtype=torch.uint8))


def norm(backward):
    f32 = torch.float32
    a = dict(q=on(1, P, T, HQ, D), k=on(1, P, T, HKV, D), gamma_q=on(1, D, dtype=f32), gamma_k=on(1, D, dtype=f32),
             cos=on(1, 9, D // 2, dtype=f32), sin=on(1, 9, D // 2, dtype=f32), pos=on(1, T, dtype=torch.int32))
    if not backward:
        return a | dict(q_out=on(1, P, T, HQ, D), k_out=on(1, P, T, HKV, D))
    return a | dict(dq_out=on(1, P, T, HQ, D), dk_out=on(1, P, T, HKV, D), dq=on(1, P, T, HQ, D), dk=on(1, P, T, HKV, D),
                    dgamma_q=on(1, P, D, dtype=f32), dgamma_k=on(1, P, D, dtype=f32), workspace=on(1, 4096, dtype=torch.uint8))


CALLS = {"attn_fwd": attention(False), "attn_bwd": attention(True), "qk_norm_rope": norm(False), "qk_norm_rope_bwd": norm(True)}


@pytest.fixture
def launched(monkeypatch):
    from ring_collectives_gb300 import _build
    _build.build()
    calls = []
    monkeypatch.setattr(rc, "_launch", lambda *a: calls.append(a))
    return calls


@pytest.mark.parametrize("call", CALLS)
def test_all_on_one_device(launched, call):
    assert set(CALLS[call]) <= set(inspect.signature(getattr(rc, call)).parameters)
    getattr(rc, call)(**CALLS[call])
    assert len(launched) == 1


@pytest.mark.parametrize("call,name", [(c, n) for c, a in CALLS.items() for n in a])
def test_one_on_another_device(launched, call, name):
    args = dict(CALLS[call])
    t = args[name]
    args[name] = on(0, *t.shape, dtype=t.dtype)
    with pytest.raises((TypeError, ValueError), match="q" if name == "q" else name):
        getattr(rc, call)(**args)
    assert not launched


@pytest.mark.parametrize("call,name", [(c, n) for c, a in CALLS.items() for n in a])
def test_one_on_the_host(launched, call, name):
    args = dict(CALLS[call])
    args[name] = torch.zeros(args[name].shape, dtype=args[name].dtype)
    with pytest.raises((TypeError, ValueError)):
        getattr(rc, call)(**args)
    assert not launched
