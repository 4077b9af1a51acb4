"""What the paged-cache calls refuse, before anything is launched (no GPU: every call here returns an error on
the host, by the C entry's own checks or by the binding's)."""
import ctypes

import pytest
import torch

import compressed_sparse_attention_attn_gb300 as csa
from compressed_sparse_attention_attn_gb300 import _abi, _build


@pytest.fixture(scope="module")
def L():
    _build.build()
    return csa.lib()


A = 4096  # stands for a device address; nothing is read: every call below is refused


def paged(**kw):
    d = dict(k=A, v=A, k_page=2048, k_row=128, k_head=64, v_page=2048, v_row=128, v_head=64, n_pages=4, page=16,
             kv_heads=2, head_dim=64)
    d.update(kw)
    return _abi.Paged(*[d[f] for f, _ in _abi.Paged._fields_])


STEP = dict(new_len=A, R=2, page=16, length=A, table=A, width=4, free=A, n_pages=8, state=A, req=A, pos=A, slot=A, N=4, cu=A,
            length_out=A, state_out=A, info=A, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(new_len=None), -1), (dict(length=None), -1), (dict(table=None), -1), (dict(free=None), -1), (dict(state=None), -1),
    (dict(req=None), -1), (dict(slot=None), -1), (dict(length_out=None), -1), (dict(state_out=None), -1), (dict(info=None), -1),
    (dict(R=0), -2), (dict(R=14001), -2), (dict(page=0), -1), (dict(n_pages=0), -1), (dict(width=0), -1), (dict(N=-1), -1),
    (dict(n_pages=1 << 28), -1), (dict(width=1 << 28), -1), (dict(N=1 << 30), -1)])
def test_page_step_refuses(L, change, code):
    assert L.csa_page_step(*{**STEP, **change}.values()) == code
    assert b"csa_page_step" in L.attn_v41_last_error()


NORM = dict(ctx=A, q=A, q_t=256, q_h=64, k=A, k_t=128, k_h=64, v=A, v_t=128, v_h=64, N=3, H=4, cache={}, pos=A, slot=A,
            q_norm=A, k_norm=A, eps=1e-6, tab=A, tab_rows=8, rd=64, at=0, half=0, q_out=A, o_t=256, o_h=64, stream=None)
CACHE = [(dict(k=None), -1), (dict(k=A + 8), -1), (dict(v=A + 2), -1), (dict(n_pages=0), -1), (dict(page=0), -1),
         (dict(kv_heads=0), -1), (dict(head_dim=0), -1), (dict(head_dim=60), -1), (dict(k_row=100), -1),
         (dict(v_head=-64), -1), (dict(n_pages=1 << 28), -1)]


@pytest.mark.parametrize("change,code", [
    (dict(ctx=None), -1), (dict(k=None), -1), (dict(pos=None), -1), (dict(v=None), -1), (dict(q_out=None), -1),
    (dict(tab=None), -1), (dict(tab_rows=0), -1), (dict(rd=63), -1), (dict(rd=-2), -1), (dict(at=1), -1), (dict(at=2), -1),
    (dict(at=-2), -1), (dict(H=0), -1), (dict(N=-1), -1), (dict(q=A + 8), -1), (dict(q_out=A + 2), -1), (dict(q_t=250), -1),
    (dict(k_h=-64), -1), (dict(o_h=3), -1), (dict(tab=A + 4), -1), (dict(slot=None, N=65), -2)]
    + [(dict(cache=c), code) for c, code in CACHE] + [(dict(cache=dict(head_dim=1032)), -1)])
def test_qk_norm_rope_refuses(L, change, code):
    a = {**NORM, **change}
    c = paged(**a["cache"])
    a["cache"] = ctypes.byref(c)
    assert L.csa_qk_norm_rope(*a.values()) == code
    assert b"csa_qk_norm_rope" in L.attn_v41_last_error()


ATTN = dict(ctx=A, q=A, q_t=256, N=3, H=4, cache={}, table=A, R=3, width=2, req=None, pos=A, sink=None, scale=0.1, window=0,
            o=A, o_t=256, lse=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(ctx=None), -1), (dict(q=None), -1), (dict(table=None), -1), (dict(pos=None), -1), (dict(o=None), -1), (dict(N=-1), -1),
    (dict(H=0), -1), (dict(H=5), -1), (dict(H=65536), -1), (dict(R=0), -1), (dict(width=0), -1), (dict(width=1 << 28), -1),
    (dict(window=-1), -1), (dict(N=4), -2), (dict(q=A + 8), -1), (dict(o=A + 2), -1), (dict(q_t=252), -1), (dict(o_t=248), -1),
    (dict(cache=dict(head_dim=264), q_t=2048, o_t=2048), -6), (dict(cache=dict(head_dim=520, v=None), q_t=4096, o_t=4096), -6)]
    + [(dict(cache=c), code) for c, code in CACHE])
def test_paged_attn_refuses(L, change, code):
    a = {**ATTN, **change}
    c = paged(**a["cache"])
    a["cache"] = ctypes.byref(c)
    assert L.csa_paged_attn(*a.values()) == code
    assert b"csa_paged_attn" in L.attn_v41_last_error()


@pytest.mark.parametrize("change", [
    dict(o_t=0), dict(o_h=0), dict(o_h=56), dict(o_t=248), dict(o_t=64), dict(cache=dict(k_head=0)), dict(cache=dict(v_head=0)),
    dict(cache=dict(k_row=64)), dict(cache=dict(k_page=1024)), dict(cache=dict(v_page=2040)),
    dict(cache=dict(k_row=64, k_head=960, k_page=2048))])
def test_qk_norm_rope_refuses_rows_that_overlap(L, change):
    a = {**NORM, **change}
    c = paged(**a["cache"])
    a["cache"] = ctypes.byref(c)
    assert L.csa_qk_norm_rope(*a.values()) == -1
    assert b"overlap" in L.attn_v41_last_error()


def test_the_binding_refuses_what_is_not_on_the_gpu():
    t = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        csa.PagedCache(t)
    with pytest.raises(ValueError, match="CUDA"):
        csa._rows(torch.zeros(2, 4, 64, dtype=torch.bfloat16), 0, "q")
    with pytest.raises(ValueError, match="CUDA"):
        csa._vec(torch.zeros(4, dtype=torch.int32), 4, torch.int32, 0, "pos")


class OnDevice:
    """Stands for a CUDA tensor: what the binding asks of one, and no memory."""
    is_cuda, dtype, shape = True, torch.bfloat16, torch.Size((4, 16, 2, 64))

    def __init__(self, index):
        self.index, self.device = index, torch.device("cuda", index)

    def dim(self):
        return 4

    def stride(self, i=None):
        s = (2048, 128, 64, 1)
        return s if i is None else s[i]

    def get_device(self):
        return self.index

    def data_ptr(self):
        return A


def test_the_binding_refuses_a_cache_over_two_devices():
    assert csa.PagedCache(OnDevice(1), OnDevice(1)).device == 1
    for k, v in ((0, 1), (1, 0)):
        with pytest.raises(ValueError, match="v: expected on cuda:%d" % k):
            csa.PagedCache(OnDevice(k), OnDevice(v))
