"""CPU checks of the serving entry points (include/jf_serving.h): both builds export what the header declares, and bad
arguments are rejected on the host before any CUDA call (so these run without a GPU)."""
import pytest
import torch

from tree_verify_attention_jf_b200 import _lib, api

BAD, UNSUP, OK = _lib.JF_ERR_INVALID_ARG, _lib.JF_ERR_UNSUPPORTED, _lib.JF_OK


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def test_both_builds_export_every_declared_symbol(L):
    names = _lib.declared_functions(_lib.SERVING_HEADER)
    assert {"jf_sample", "jf_accept_sampled"} <= set(names)
    for n in names:
        assert hasattr(L, n) and hasattr(_lib.debug_lib(), n), n


def test_sample_host_validation(L):
    # the valid call has no rows, so nothing is ever launched; with rows, a null pointer stops the call
    def call(**o):
        a = dict(x=None, ty=0, stride=1000, R=0, V=1000, u=8, t=8, tok=8)
        a.update(o)
        return L.jf_sample(a["x"], a["ty"], a["stride"], a["R"], a["V"], a["u"], a["t"], None, None, None, a["tok"],
                           None, None, None)
    assert call() == OK
    assert call(R=3) == BAD                       # null logits
    assert call(R=3, x=24) == BAD                 # not 16-byte aligned
    for null in ("u", "t", "tok"):
        assert call(R=3, x=16, **{null: None}) == BAD
    for bad in (dict(R=-1), dict(V=0), dict(V=-4), dict(stride=999), dict(ty=2), dict(ty=-1)):
        assert call(**bad) == BAD, bad
    assert call(V=524289, stride=600000) == UNSUP
    assert call(R=(1 << 24) + 1) == UNSUP


def test_accept_sampled_host_validation(L):
    def call(**o):
        a = dict(tok=8, par=8, x=None, ty=0, u=8, t=8, B=0, N=16, V=1000, D=4, acc=8, path=8, bonus=8)
        a.update(o)
        return L.jf_accept_sampled(a["tok"], a["par"], a["x"], a["ty"], a["u"], a["t"], None, None, None, a["B"],
                                   a["N"], a["V"], a["D"], a["acc"], a["path"], a["bonus"], None, None, None)
    assert call() == OK
    assert call(B=2) == BAD
    assert call(B=2, x=24) == BAD
    for null in ("tok", "par", "u", "t", "acc", "path", "bonus"):
        assert call(B=2, x=16, **{null: None}) == BAD
    for bad in (dict(B=-1), dict(N=0), dict(V=0), dict(D=-1), dict(ty=7)):
        assert call(**bad) == BAD, bad
    for big in (dict(N=1025), dict(D=1024), dict(V=524289), dict(B=(1 << 24) + 1)):
        assert call(**big) == UNSUP, big


def test_python_calls_refuse_cpu_tensors():
    x, u, t = torch.zeros(2, 8), torch.zeros(2), torch.ones(2)
    with pytest.raises(ValueError, match="CUDA"):
        api.sample(x, u, t)
    i = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        api.accept_sampled(i, i, torch.zeros(2, 3, 8), torch.zeros(2, 5), t, 4)
