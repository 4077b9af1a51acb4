"""What prompt_attn and prefix_attn refuse, before anything is launched (no GPU: every call here returns an error on the host)."""
import ctypes

import pytest

from test_paged_refusals import A, CACHE, L, paged  # noqa: F401

PROMPT = dict(ctx=A, q=A, q_t=256, N=3, H=4, cache={}, table=A, R=3, width=2, cu=A, length=A, sink=None, scale=0.1, window=0, o=A,
              o_t=256, lse=None, stream=None)
PREFIX = dict(ctx=A, q=A, q_t=256, N=3, H=4, cache={}, table=A, R=3, width=2, req=None, pos=A, prefix=A, G=2, prefix_width=2,
              prefix_len=A, cu=A, sink=None, scale=0.1, window=0, o=A, o_t=256, lse=None, stream=None)
ALIKE = [(dict(ctx=None), -1), (dict(q=None), -1), (dict(table=None), -1), (dict(o=None), -1), (dict(N=-1), -1), (dict(H=0), -1),
         (dict(H=5), -1), (dict(H=65536), -1), (dict(R=0), -1), (dict(width=0), -1), (dict(width=1 << 28), -1), (dict(window=-1), -1),
         (dict(q=A + 8), -1), (dict(o=A + 2), -1), (dict(q_t=252), -1), (dict(o_t=248), -1), (dict(q_t=260), -1),
         (dict(cache=dict(head_dim=264), q_t=2048, o_t=2048), -6), (dict(cache=dict(head_dim=512, v=None), q_t=4096, o_t=4096), -6),
         (dict(N=1 << 29), -2)] + [(dict(cache=c), code) for c, code in CACHE]


def call(f, args, change):
    a = {**args, **change}
    c = paged(**a["cache"])
    a["cache"] = ctypes.byref(c)
    return f(*a.values())


@pytest.mark.parametrize("change,code", ALIKE + [(dict(cu=None), -1), (dict(length=None), -1)])
def test_prompt_attn_refuses(L, change, code):  # noqa: F811
    assert call(L.csa_prompt_attn, PROMPT, change) == code
    assert b"csa_prompt_attn" in L.attn_v41_last_error()


@pytest.mark.parametrize("change,code", ALIKE + [
    (dict(pos=None), -1), (dict(prefix=None), -1), (dict(prefix_len=None), -1), (dict(cu=None), -1), (dict(G=0), -1),
    (dict(prefix_width=0), -1), (dict(prefix_width=1 << 28), -1), (dict(N=4), -2)])
def test_prefix_attn_refuses(L, change, code):  # noqa: F811
    assert call(L.csa_prefix_attn, PREFIX, change) == code
    assert b"csa_prefix_attn" in L.attn_v41_last_error()


def test_the_bindings_shapes():
    """What the Python calls refuse before the C entry (stand-ins for CUDA tensors that hold no memory)."""
    import torch

    import compressed_sparse_attention_attn_gb300 as csa

    class T:
        def __init__(self, shape, dtype, strides=None):
            self.shape, self.dtype, self.device, self.s = torch.Size(shape), dtype, torch.device("cuda", 0), strides

        def dim(self):
            return len(self.shape)

        def stride(self, i=None):
            if self.s is None:
                self.s = [1] * len(self.shape)
                for k in range(len(self.shape) - 2, -1, -1):
                    self.s[k] = self.s[k + 1] * self.shape[k + 1]
            return tuple(self.s) if i is None else self.s[i]

        def get_device(self):
            return 0

        def numel(self):
            return self.shape.numel()

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return A

    class Cache:
        head_dim, kv_heads, device, ref = 64, 2, 0, None

    class Ctx(csa.Context):
        def __init__(self):
            self.h = None

    bf, i32 = torch.bfloat16, torch.int32
    q, out = T((3, 4, 64), bf), T((3, 4, 64), bf)
    ctx, stream = Ctx(), T((1,), i32)
    stream.cuda_stream = 0
    now, csa._now = csa._now, lambda s: (0, 0)
    try:
        good = dict(q=q, cache=Cache, table=T((2, 5), i32), cu=T((3,), i32), length=T((2,), i32), scale=0.1, out=out, stream=stream)
        for change in (dict(q=T((3, 4, 72), bf)), dict(table=T((10,), i32)), dict(out=T((3, 4, 32), bf)), dict(cu=T((2,), i32)),
                       dict(cu=T((3,), torch.int64)), dict(length=T((3,), i32)), dict(q=T((3, 4, 64), torch.float16)),
                       dict(lse=T((3, 3), torch.float32)), dict(sink=T((5,), torch.float32)), dict(q=T((3, 4, 64), bf, [512, 128, 1])),
                       dict(q=T((3, 4, 64), bf, [512, 64, 2]))):
            with pytest.raises(ValueError):
                ctx.prompt_attn(**{**good, **change})
        good = dict(q=q, cache=Cache, table=T((3, 5), i32), pos=T((3,), i32), prefix=T((2, 4), i32), prefix_len=T((2,), i32),
                    scale=0.1, cu=T((3,), i32), out=out, stream=stream)
        for change in (dict(pos=T((2,), i32)), dict(prefix=T((8,), i32)), dict(prefix_len=T((1,), i32)), dict(cu=T((2,), i32)),
                       dict(req=T((2,), i32)), dict(prefix=T((2, 4), torch.int64)), dict(q=T((3, 4, 72), bf))):
            with pytest.raises(ValueError):
                ctx.prefix_attn(**{**good, **change})
    finally:
        csa._now = now
