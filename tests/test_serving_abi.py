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
    assert set(names) == {"jf_sample", "jf_accept_sampled", "jf_tree_attention_shared_workspace_size",
                          "jf_tree_attention_shared", "jf_tree_attention_shared_fp8"}
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


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_shared_host_validation(L, fp8):
    # the valid call has no nodes, so nothing is ever launched; with nodes, a null or short argument stops the call
    def call(**o):
        a = dict(q=16, k=32, v=48, ks=0.1, vs=0.1, bt=64, maxp=4, pl=64, to=64, par=64, go=64, sl=64, G=2, B=3, T=0, hq=4,
                 hkv=1, d=128, page=16, pages=8, scale=0.1, out=64, ws=256,
                 wsb=L.jf_tree_attention_shared_workspace_size(10, 4))
        a.update(o)
        fn = L.jf_tree_attention_shared_fp8 if fp8 else L.jf_tree_attention_shared
        return fn(a["q"], a["k"], a["v"], *((a["ks"], a["vs"]) if fp8 else ()), a["bt"], a["maxp"], a["pl"], a["to"],
                  a["par"], a["go"], a["sl"], a["G"], a["B"], a["T"], a["hq"], a["hkv"], a["d"], a["page"], a["pages"],
                  a["scale"], a["out"], None, a["ws"], a["wsb"], None, None)
    assert call() == OK
    assert call(B=0, G=0, T=5) == OK
    for null in ("q", "k", "v", "bt", "pl", "to", "par", "go", "sl", "out", "ws"):
        assert call(T=10, **{null: None}) == BAD, null
    for bad in (dict(G=-1), dict(G=4), dict(G=0, T=10), dict(scale=0.0), dict(hkv=0), dict(T=10, q=24),
                dict(T=10, ws=257), dict(T=10, wsb=100), dict(T=11)):
        assert call(**bad) == BAD, bad
    for bad in (dict(d=64), dict(page=32), dict(hq=6, hkv=4), dict(B=1000, G=25), dict(pages=1 << 27)):
        assert call(**bad) == UNSUP, bad
    if fp8:
        assert call(ks=0.0) == BAD and call(vs=float("nan")) == BAD
    size = L.jf_tree_attention_shared_workspace_size
    assert size(10, 4) < size(11, 4) < size(11, 32) and size(10, 4) % 256 == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_shared_refuses_counts_whose_sum_passes_32_bits(L, fp8):
    # no nodes: nothing is launched even where the call is taken
    fn = L.jf_tree_attention_shared_fp8 if fp8 else L.jf_tree_attention_shared
    for B, G in ((2 ** 31 - 1, 1), (2 ** 30, 2 ** 30), (2 ** 31 - 1, 2 ** 31 - 1)):
        assert fn(16, 32, 48, *((0.1, 0.1) if fp8 else ()), 64, 4, 64, 64, 64, 64, 64, G, B, 0, 4, 1, 128, 16, 8, 0.1,
                  64, None, 256, 1 << 40, None, None) == UNSUP


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_shared_refuses_tables_of_more_slots_than_32_bits_count(L, fp8):
    # a prefix of almost 2^31 slots fits such a table, and its tiles would be counted in 32 bits; no nodes, as above
    fn = L.jf_tree_attention_shared_fp8 if fp8 else L.jf_tree_attention_shared
    for pages, want in (((1 << 27) - 16, OK), ((1 << 27) - 15, UNSUP), (1 << 27, UNSUP), (2 ** 31 - 1, UNSUP)):
        assert fn(16, 32, 48, *((0.1, 0.1) if fp8 else ()), 64, pages, 64, 64, 64, 64, 64, 1, 3, 0, 4, 1, 128, 16, 8, 0.1,
                  64, None, 256, 1 << 40, None, None) == want, pages


def test_python_calls_refuse_cpu_tensors():
    x, u, t = torch.zeros(2, 8), torch.zeros(2), torch.ones(2)
    with pytest.raises(ValueError, match="CUDA"):
        api.sample(x, u, t)
    i = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        api.accept_sampled(i, i, torch.zeros(2, 3, 8), torch.zeros(2, 5), t, 4)
