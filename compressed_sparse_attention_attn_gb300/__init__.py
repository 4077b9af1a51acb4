"""GB300 (sm_103a) compressed sparse attention layer core of DeepSeek-V4.1.

Python face of the C ABI in ``include/csa.h``: every function here marshals torch CUDA tensors
(device pointers, the current stream) into one library call; all arithmetic runs in the library's
CUDA kernels.  bf16 tensors are ``torch.bfloat16``; int8/uint8/int32/f32 as the header states.
"""
import ctypes

import torch

from . import _abi

_lib = None


def lib():
    global _lib
    if _lib is None:
        _lib = _abi.load()
    return _lib


class CsaError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        msg = lib().attn_v41_last_error().decode(errors="replace")
        super().__init__("%s: %s (%s)" % (where, _abi.ERRORS.get(code, code), msg))


def _check(rc, where):
    if rc != 0:
        raise CsaError(rc, where)


def _checked(t, dtype, cuda, what):
    if t.is_cuda != cuda:
        raise ValueError("%s: expected a %s tensor, got one on %s" % (what, "CUDA" if cuda else "host", t.device))
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s: expected %s, got %s" % (what, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s: expected a contiguous tensor (shape %s, strides %s)" % (what, tuple(t.shape), t.stride()))
    return ctypes.c_void_p(t.data_ptr())


def _dev(t, dtype=None, what="tensor"):
    """Device pointer of a contiguous CUDA tensor of the given dtype; None -> NULL.  The kernels read
    and write through raw pointers, so a host tensor, a strided view or a narrower dtype is refused
    here rather than read out of bounds on the GPU."""
    return None if t is None else _checked(t, dtype, True, what)


def _host(t, dtype=None, what="tensor"):
    """Host pointer of a contiguous CPU tensor of the given dtype (pinned for copies that overlap)."""
    return None if t is None else _checked(t, dtype, False, what)


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _empty(shape, dtype, device, stream):
    """A tensor that belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _now(stream):
    """(current device, raw stream) of a call; looked up once a call, without building a Stream object."""
    dev = torch._C._cuda_getDevice()
    return dev, (torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)


def _rows(t, dev, what):
    """(pointer, token stride, head stride) of a bf16 tensor [N, heads, hd] on CUDA device dev whose features are
    contiguous."""
    if t.get_device() != dev or t.dtype is not torch.bfloat16:
        raise ValueError("%s: expected a bfloat16 tensor on the current CUDA device, got %s on %s" % (what, t.dtype, t.device))
    s0, s1, s2 = t.stride()
    n, h, d = t.shape
    if s2 != 1 and d > 1:
        raise ValueError("%s: the features of a head must be contiguous (strides %s)" % (what, t.stride()))
    if h == 1:
        s1 = d
    if n <= 1:
        s0 = s1 * h
    return t.data_ptr(), s0, s1


def _vec(t, n, dtype, dev, what):
    """Pointer of a contiguous tensor of n values on CUDA device dev; None -> NULL."""
    if t is None:
        return None
    if t.get_device() != dev or t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError("%s: expected a contiguous tensor of %d %s on the current CUDA device, got %s %s on %s" % (
            what, n, dtype, tuple(t.shape), t.dtype, t.device))
    return t.data_ptr()


class PagedCache:
    """A csa_paged: pages of key rows k [n_pages, page, kv_heads, hd] and value rows v alike (None: the key rows are
    the values), bf16 CUDA tensors or views of either order of rows and heads (the features contiguous)."""

    def __init__(self, k, v=None):
        for t, what in ((k, "k"), (v, "v")):
            if t is None and what == "v":
                continue
            if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 4 or t.shape != k.shape or t.stride(3) != 1:
                raise ValueError("%s: expected a CUDA bfloat16 tensor [n_pages, page, kv_heads, hd] with contiguous "
                                 "features, got %s %s, strides %s on %s" % (what, tuple(t.shape), t.dtype, t.stride(), t.device))
        if v is not None and v.device != k.device:
            raise ValueError("v: expected on %s as k is, got one on %s" % (k.device, v.device))
        self.k, self.v = k, v
        self.n_pages, self.page, self.kv_heads, self.head_dim = k.shape
        st = lambda t: [0 if t.shape[i] == 1 else t.stride(i) for i in range(3)]  # noqa: E731
        self.c = _abi.Paged(k.data_ptr(), None if v is None else v.data_ptr(), *st(k), *(st(v) if v is not None else (0, 0, 0)),
                            *k.shape)
        self.ref = ctypes.byref(self.c)
        self.device = k.get_device()


CFG_FIELDS = [f for f, _ in _abi.Cfg._fields_]


def make_cfg(geom):
    """csa_cfg from a mapping (or an object with the same attribute names)."""
    get = geom.get if isinstance(geom, dict) else (lambda k, d=None: getattr(geom, k, d))
    vals = {}
    for f, ty in _abi.Cfg._fields_:
        v = get(f, 0)
        vals[f] = float(v) if ty is _abi.F else int(v)
    return _abi.Cfg(**vals)


def make_role(role):
    return _abi.Role(int(role.get("ratio", 0)), int(role.get("is_kv_source", 0)), int(role.get("is_index_source", 0)),
                     int(role.get("is_candidate_source", 0)), int(role.get("uses_candidates", 0)))


class Shared:
    """What source layers publish (SharedV41 of the attn_v41 runtime) as device tensors."""

    def __init__(self, compress_kv, index_k, compress_len, topk_idxs, topk, candidates=None, has_topk=False):
        self.compress_kv = compress_kv
        self.index_k = index_k
        self.compress_len = int(compress_len)
        self.topk_idxs = topk_idxs
        self.topk = int(topk)
        self.candidates = candidates
        self.has_topk = bool(has_topk)
        self._c = None

    def struct(self):
        stride = self.compress_kv.shape[1] if self.compress_kv is not None else 0
        self._c = _abi.Shared(_dev(self.compress_kv, torch.bfloat16, "compress_kv"), _dev(self.index_k, torch.bfloat16, "index_k"),
                              self.compress_len, stride, _dev(self.topk_idxs, torch.int32, "topk_idxs"), self.topk,
                              int(self.has_topk), _dev(self.candidates, torch.uint8, "candidates"),
                              0 if self.candidates is None else self.candidates.shape[-1])
        return self._c

    def sync_back(self, kv_state=None, with_keys=False):
        """What the library published into the struct: the selection flag and, after a kv source (its
        kv_state), its caches and their length."""
        if self._c is not None:
            self.has_topk = bool(self._c.has_topk)
            self.compress_len = int(self._c.compress_len)
        if kv_state is not None:
            self.compress_kv = kv_state["latent"]
            if with_keys:
                self.index_k = kv_state["index_keys"]


DEBUG_FIELDS = ("q", "kv", "kv_codes", "kv_scale", "idx", "scores", "o", "og", "qr", "qI", "wI")
DEBUG_DTYPES = (torch.bfloat16, torch.bfloat16, torch.uint8, torch.int8, torch.int32, torch.float32, torch.bfloat16, torch.bfloat16, torch.bfloat16, torch.bfloat16, torch.float32)
WEIGHT_FIELDS = ("sink", "q_norm", "kv_norm", "wq_a", "wq_b", "wkv", "wo_a", "wo_b", "idx_wq_b", "idx_wproj",
                 "wo_a_fp8", "wo_a_scale", "comp_wkv", "comp_wgate", "comp_norm", "idx_wk", "idx_k_norm")
# (comp_wkv is f32 at ratio > 1 and bf16 at ratio 1: its dtype is checked against the role)
WEIGHT_DTYPES = (torch.float32, torch.float32, torch.float32, torch.bfloat16, torch.bfloat16, torch.bfloat16, torch.bfloat16,
                 torch.bfloat16, torch.bfloat16, torch.bfloat16, torch.uint8, torch.float32, None, torch.float32,
                 torch.float32, torch.bfloat16, torch.float32)


def make_state(ring, kv_state=None):
    """csa_layer_state: the window ring, and for a kv source the dict kv_state with comp_kv,
    comp_score (f32 [max_batch, ratio, hd]), latent (bf16 [max_batch, rows, hd]) and index_keys (bf16
    [max_batch, rows, index_hd], may be None)."""
    if kv_state is None:
        return _abi.LayerState(_dev(ring, torch.bfloat16, "ring"))
    kv, sc, lat = kv_state["comp_kv"], kv_state["comp_score"], kv_state["latent"]
    ik = kv_state.get("index_keys")
    return _abi.LayerState(_dev(ring, torch.bfloat16, "ring"), _dev(kv, torch.float32, "comp_kv"),
                           _dev(sc, torch.float32, "comp_score"), kv.shape[1], _dev(lat, torch.bfloat16, "latent"),
                           _dev(ik, torch.bfloat16, "index_keys"), lat.shape[1])


class Context:
    """A csa_ctx: workspaces and RoPE tables for one geometry, on the current CUDA device."""

    def __init__(self, geom):
        self.geom = geom
        self.cfg = make_cfg(geom)
        h = ctypes.c_void_p()
        _check(lib().csa_create(ctypes.byref(self.cfg), ctypes.byref(h)), "csa_create")
        self.h = h

    def close(self):
        if getattr(self, "h", None) is not None and self.h.value:
            lib().csa_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- layer ---------------------------------------------------------------------------------
    @staticmethod
    def layer_weights(w, role):
        wkv = w.get("comp_wkv")
        if wkv is not None:
            want = torch.float32 if int(role.get("ratio", 0)) > 1 else torch.bfloat16
            _dev(wkv, want, "comp_wkv")
        return _abi.LayerWeights(make_role(role), *[_dev(w.get(n), dt, n) for n, dt in zip(WEIGHT_FIELDS, WEIGHT_DTYPES)])

    def state_init(self, ring, batch, stream=None, kv_state=None):
        st = make_state(ring, kv_state)
        _check(lib().csa_state_init(self.h, ctypes.byref(st), batch, _stream(stream)), "csa_state_init")

    def compress(self, w, role, ring, kv_state, x, start_pos, shared=None, y_dbg=None, stream=None):
        """csa_compress: the kv source's compressor over x [B, T, dim]; publishes into shared."""
        B, T, _ = x.shape
        lw = self.layer_weights(w, role)
        st = make_state(ring, kv_state)
        sh = shared.struct() if shared is not None else None
        _check(lib().csa_compress(self.h, ctypes.byref(lw), ctypes.byref(st), _dev(x, torch.bfloat16, "x"), B, T,
                                  start_pos, ctypes.byref(sh) if sh is not None else None,
                                  _dev(y_dbg, torch.bfloat16, "y_dbg"), _stream(stream)), "csa_compress")
        if shared is not None:
            shared.sync_back(kv_state, w.get("idx_wk") is not None)

    def forward(self, w, role, ring, x, start_pos, shared=None, out=None, debug=None, stream=None, lw=None,
                kv_state=None):
        """attn_v41_forward.  x [B, T, dim] bf16 -> out [B, T, dim] bf16; ring [max_batch, W, hd] bf16.
        ``debug``: dict of preallocated device tensors named as in csa_debug.  ``lw``: a prebuilt
        LayerWeights struct (skips re-marshalling)."""
        B, T, _ = x.shape
        if out is None:
            out = torch.empty_like(x)
        if lw is None:
            lw = self.layer_weights(w, role)
        st = make_state(ring, kv_state)
        sh = shared.struct() if shared is not None else None
        dbg = None
        if debug:
            dbg = _abi.Debug(*[_dev(debug.get(n), dt, n) for n, dt in zip(DEBUG_FIELDS, DEBUG_DTYPES)])
        rc = lib().attn_v41_forward(self.h, ctypes.byref(lw), ctypes.byref(st), _dev(x, torch.bfloat16, "x"), B, T, start_pos,
                                    ctypes.byref(sh) if sh is not None else None, _dev(out, torch.bfloat16, "out"),
                                    ctypes.byref(dbg) if dbg is not None else None, _stream(stream))
        _check(rc, "attn_v41_forward")
        if shared is not None:
            shared.sync_back(kv_state if int(role.get("is_kv_source", 0)) else None, bool(lw.idx_wk))
        return out

    def forward_host(self, lw, ring, x_host, start_pos, shared, out_host, B, T, stream=None):
        """attn_v41_forward_host with host tensors (pinned for overlap)."""
        st = _abi.LayerState(_dev(ring, torch.bfloat16, "ring"))
        sh = shared.struct() if shared is not None else None
        rc = lib().attn_v41_forward_host(self.h, ctypes.byref(lw), ctypes.byref(st), _host(x_host, torch.bfloat16, "x_host"), B, T,
                                         start_pos, ctypes.byref(sh) if sh is not None else None,
                                         _host(out_host, torch.bfloat16, "out_host"), _stream(stream))
        _check(rc, "attn_v41_forward_host")
        if shared is not None:
            shared.sync_back()

    def rope_table(self, ratio_class):
        g = self.cfg
        t = torch.empty(g.max_seq, g.rope_dim // 2, 2, dtype=torch.float32)
        _check(lib().csa_rope_table_get(self.h, ratio_class, _host(t, torch.float32, "table")), "csa_rope_table_get")
        return t

    def status(self, clear=True):
        return lib().csa_status(self.h, int(clear))

    def workspace_bytes(self):
        return lib().csa_workspace_bytes(self.h)

    def trace(self, enable=True, append=False):
        """Stage tracing: enable (each forward lists its own stages) or, with append, every forward
        appends to one list that restarts here (several layers, or a captured and replayed step)."""
        _check(lib().csa_trace_enable(self.h, 2 if (enable and append) else int(bool(enable))), "csa_trace_enable")

    def trace_read(self):
        """[(stage name, milliseconds)] of the listed stages (waits for their events)."""
        names = (ctypes.c_char_p * 64)()
        ms = (ctypes.c_float * 64)()
        n = lib().csa_trace_read(self.h, 64, names, ms)
        if n < 0:
            _check(n, "csa_trace_read")
        return [(names[i].decode(), float(ms[i])) for i in range(min(n, 64))]

    def last_launches(self):
        return lib().csa_last_launches(self.h)

    # -- steps ---------------------------------------------------------------------------------
    def linear(self, x, W, out=None, groups=1, stream=None):
        """y = x W^T (bf16, f32 accumulation); groups > 1: block-diagonal W [groups*N, K]."""
        K = W.shape[1]
        N = W.shape[0] // groups
        M = x.numel() // x.shape[-1]
        if out is None:
            out = torch.empty(x.shape[:-1] + (N * groups,), dtype=torch.bfloat16, device=x.device)
        _check(lib().csa_linear(self.h, _dev(x, torch.bfloat16, "x"), M, K, x.shape[-1], _dev(W, torch.bfloat16, "W"), N, K, _dev(out, torch.bfloat16, "out"),
                                out.shape[-1], groups, _stream(stream)), "csa_linear")
        return out

    def linear_fp8w(self, x, W8, scale, out=None, groups=1, stream=None):
        """y = x w^T with w = bf16(e4m3(W8) * scale per 128 x 128 tile); W8 uint8 [groups*N, K] codes,
        scale f32 [ceil(groups*N/128), ceil(K/128)]."""
        K = W8.shape[1]
        N = W8.shape[0] // groups
        M = x.numel() // x.shape[-1]
        if out is None:
            out = torch.empty(x.shape[:-1] + (N * groups,), dtype=torch.bfloat16, device=x.device)
        _check(lib().csa_linear_fp8w(self.h, _dev(x, torch.bfloat16, "x"), M, K, x.shape[-1], _dev(W8, torch.uint8, "W8"),
                                     _dev(scale, torch.float32, "scale"), N, K, _dev(out, torch.bfloat16, "out"),
                                     out.shape[-1], groups, _stream(stream)), "csa_linear_fp8w")
        return out

    def sparse_attn(self, q, rows_a, a_len, idx_a, sink, scale, rows_b=None, b_len=0, idx_b=None, o=None, o_rot=None,
                    rd=0, start_pos=0, tab=None, B=1, T=None, stream=None):
        """q [B*T, H, hd]; rows_a [B, ., hd]; rows_b [B, ., hd]; idx_a [B*T, na]; idx_b [B*T, nb]."""
        n, H, hd = q.shape
        T = n // B if T is None else T
        _check(lib().csa_sparse_attn(self.h, _dev(q, torch.bfloat16, "q"), B, T, H, hd, _dev(rows_a, torch.bfloat16, "rows_a"),
                                     rows_a.shape[1] * hd, a_len, _dev(rows_b, torch.bfloat16, "rows_b"),
                                     0 if rows_b is None else rows_b.shape[1] * hd, b_len, _dev(idx_a, torch.int32, "idx_a"),
                                     idx_a.shape[1], _dev(idx_b, torch.int32, "idx_b"), 0 if idx_b is None else idx_b.shape[1],
                                     _dev(sink, torch.float32, "sink"), scale, _dev(o, torch.bfloat16, "o"), _dev(o_rot, torch.bfloat16, "o_rot"), rd,
                                     start_pos, _dev(tab, torch.float32, "tab"), 0 if tab is None else tab.shape[0],
                                     _stream(stream)), "csa_sparse_attn")


    # -- a continuous batch over a paged cache ---------------------------------------------------
    def qk_norm_rope(self, q, k, v, cache, pos, slot=None, tab=None, rd=0, rope_at=None, half=False, q_norm=None,
                     k_norm=None, eps=None, q_out=None, stream=None):
        """csa_qk_norm_rope: RMSNorm (q_norm, k_norm f32 [hd] or None) of each head of q [N, H, hd] and
        k [N, kv_heads, hd], rotation of the rd features from rope_at (default: the last rd) by the angles
        tab[pos] (adjacent pairs, or with half pairs rd / 2 apart), key and value rows written to rows slot of
        the PagedCache.  q, k, v may be strided views (of a fused projection, say); q may be None, v too where
        the cache has no values.  pos, slot int32 [N]; pos < 0: a padding row, left as it is; slot -1: no
        cache row.  Returns q_out (allocated unless given; q itself for in place)."""
        N, Hk, hd = k.shape
        dev, st = _now(stream)
        if Hk != cache.kv_heads or hd != cache.head_dim:
            raise ValueError("k: expected [N, %d, %d], got %s" % (cache.kv_heads, cache.head_dim, tuple(k.shape)))
        if cache.device != dev:
            raise ValueError("cache: on CUDA device %d, the current one is %d" % (cache.device, dev))
        H = 0
        qp = op = vp = tp = None
        q_t = q_h = o_t = o_h = v_t = v_h = rows = 0
        if q is not None:
            if q.dim() != 3 or q.shape[0] != N or q.shape[2] != hd:
                raise ValueError("q: expected [%d, H, %d], got %s" % (N, hd, tuple(q.shape)))
            H = q.shape[1]
            if q_out is None:
                q_out = _empty((N, H, hd), torch.bfloat16, q.device, stream)
            elif q_out.shape != q.shape:
                raise ValueError("q_out: expected %s, got %s" % (tuple(q.shape), tuple(q_out.shape)))
            qp, q_t, q_h = _rows(q, dev, "q")
            op, o_t, o_h = _rows(q_out, dev, "q_out")
        kp, k_t, k_h = _rows(k, dev, "k")
        if cache.v is not None:
            if v is None or v.shape != k.shape:
                raise ValueError("v: expected %s, got %s" % (tuple(k.shape), None if v is None else tuple(v.shape)))
            vp, v_t, v_h = _rows(v, dev, "v")
        if tab is not None and rd:
            if tab.dim() != 3 or tab.shape[1] * 2 != rd or tab.shape[2] != 2:
                raise ValueError("tab: expected [positions, %d, 2], got %s" % (rd // 2, tuple(tab.shape)))
            rows = tab.shape[0]
            tp = _vec(tab, rows * rd, torch.float32, dev, "tab")
        _check(lib().csa_qk_norm_rope(
            self.h, qp, q_t, q_h, kp, k_t, k_h, vp, v_t, v_h, N, H, cache.ref, _vec(pos, N, torch.int32, dev, "pos"),
            _vec(slot, N, torch.int32, dev, "slot"), _vec(q_norm, hd, torch.float32, dev, "q_norm"),
            _vec(k_norm, hd, torch.float32, dev, "k_norm"), self.cfg.eps if eps is None else eps, tp, rows, rd,
            hd - rd if rope_at is None else rope_at, 1 if half else 0, op, o_t, o_h, st), "csa_qk_norm_rope")
        return q_out

    def paged_attn(self, q, cache, table, pos, scale, req=None, sink=None, window=0, out=None, lse=None,
                   with_lse=False, stream=None):
        """csa_paged_attn: row n of q [N, H, hd] (a token stride is allowed) attends rows max(0, pos[n]+1-window)
        .. pos[n] of request req[n] (None: request n) of the PagedCache through table int32 [R, width].
        pos -1: no rows (zeros); pos < -1 or req < 0: padding, its row of out is left as it is.  sink f32 [H].
        Returns out, or (out, lse) with lse f32 [N, H] the log of the sum of exponentials (without the sink)
        when lse is given or with_lse is set."""
        N, H, hd = q.shape
        dev, st = _now(stream)
        if hd != cache.head_dim:
            raise ValueError("q: expected [N, H, %d], got %s" % (cache.head_dim, tuple(q.shape)))
        if cache.device != dev:
            raise ValueError("cache: on CUDA device %d, the current one is %d" % (cache.device, dev))
        if table.dim() != 2:
            raise ValueError("table: expected [requests, width], got %s" % (tuple(table.shape),))
        R, width = table.shape
        if out is None:
            out = _empty((N, H, hd), torch.bfloat16, q.device, stream)
        elif out.shape != q.shape:
            raise ValueError("out: expected %s, got %s" % (tuple(q.shape), tuple(out.shape)))
        if lse is None and with_lse:
            lse = _empty((N, H), torch.float32, q.device, stream)
        qp, q_t, q_h = _rows(q, dev, "q")
        op, o_t, o_h = _rows(out, dev, "out")
        if H > 1 and (q_h != hd or o_h != hd):
            raise ValueError("q, out: the heads of a token must follow one another")
        _check(lib().csa_paged_attn(
            self.h, qp, q_t, N, H, cache.ref, _vec(table, R * width, torch.int32, dev, "table"), R, width,
            _vec(req, N, torch.int32, dev, "req"), _vec(pos, N, torch.int32, dev, "pos"),
            _vec(sink, H, torch.float32, dev, "sink"), scale, window, op, o_t,
            _vec(lse, N * H, torch.float32, dev, "lse"), st), "csa_paged_attn")
        return out if lse is None else (out, lse)

    def _rows_call(self, q, cache, table, what, out, lse, with_lse, stream):
        """What prompt_attn and prefix_attn marshal alike: (device, stream, out, lse, leading C arguments, trailing ones)."""
        N, H, hd = q.shape
        dev, st = _now(stream)
        if hd != cache.head_dim:
            raise ValueError("q: expected [N, H, %d], got %s" % (cache.head_dim, tuple(q.shape)))
        if cache.device != dev:
            raise ValueError("cache: on CUDA device %d, the current one is %d" % (cache.device, dev))
        if table.dim() != 2:
            raise ValueError("table: expected [%s, width], got %s" % (what, tuple(table.shape)))
        R, width = table.shape
        if out is None:
            out = _empty((N, H, hd), torch.bfloat16, q.device, stream)
        elif out.shape != q.shape:
            raise ValueError("out: expected %s, got %s" % (tuple(q.shape), tuple(out.shape)))
        if lse is None and with_lse:
            lse = _empty((N, H), torch.float32, q.device, stream)
        qp, q_t, q_h = _rows(q, dev, "q")
        op, o_t, o_h = _rows(out, dev, "out")
        if H > 1 and (q_h != hd or o_h != hd):
            raise ValueError("q, out: the heads of a token must follow one another")
        return (dev, st, out, lse, (self.h, qp, q_t, N, H, cache.ref, _vec(table, R * width, torch.int32, dev, "table"), R, width),
                (op, o_t, _vec(lse, N * H, torch.float32, dev, "lse"), st))

    def prompt_attn(self, q, cache, table, cu, length, scale, sink=None, window=0, out=None, lse=None, with_lse=False,
                    stream=None):
        """csa_prompt_attn: causal attention of each request's new tokens over the PagedCache.  Rows cu[r] .. cu[r+1]-1 of
        q [N, H, hd] (a token stride is allowed) are the newest of the length[r] rows that request r has behind table
        int32 [R, width]; cu int32 [R+1] and length int32 [R] are page_step's cu and length_out.  Decoding requests may be
        among them; a step of nothing else is faster with paged_attn.  Rows outside every request are left as they are.
        sink f32 [H].  Returns out, or (out, lse) as paged_attn does."""
        dev, st, out, lse, head, tail = self._rows_call(q, cache, table, "requests", out, lse, with_lse, stream)
        R, H, i32 = table.shape[0], q.shape[1], torch.int32
        _check(lib().csa_prompt_attn(*head, _vec(cu, R + 1, i32, dev, "cu"), _vec(length, R, i32, dev, "length"),
                                     _vec(sink, H, torch.float32, dev, "sink"), scale, window, *tail), "csa_prompt_attn")
        return out if lse is None else (out, lse)

    def prefix_attn(self, q, cache, table, pos, prefix, prefix_len, scale, cu=None, req=None, sink=None, window=0, out=None,
                    lse=None, with_lse=False, stream=None):
        """csa_prefix_attn: paged_attn for rows that share a prefix.  Row n of q [N, H, hd] attends the prefix_len[g] rows
        behind prefix int32 [G, width] of its prefix g, then rows 0 .. pos[n] of request req[n] (None: request n) behind
        table int32 [R, width]; with a window, the last `window` of them.  Prefix g is that of rows cu[g] .. cu[g+1]-1
        (cu None: one prefix for all).  pos -1: the prefix alone; pos < -1 or req < 0: padding, left as it is.
        N * H up to 330, 130, 61 and 66 thousand at 64, 128, 192 and 256 features fit the workspace; more raises CsaError.
        Returns out, or (out, lse) as paged_attn does."""
        dev, st, out, lse, head, tail = self._rows_call(q, cache, table, "requests", out, lse, with_lse, stream)
        N, H, i32 = q.shape[0], q.shape[1], torch.int32
        if prefix.dim() != 2:
            raise ValueError("prefix: expected [prefixes, width], got %s" % (tuple(prefix.shape),))
        G, width = prefix.shape
        _check(lib().csa_prefix_attn(
            *head, _vec(req, N, i32, dev, "req"), _vec(pos, N, i32, dev, "pos"), _vec(prefix, G * width, i32, dev, "prefix"), G,
            width, _vec(prefix_len, G, i32, dev, "prefix_len"), _vec(cu, G + 1, i32, dev, "cu"),
            _vec(sink, H, torch.float32, dev, "sink"), scale, window, *tail), "csa_prefix_attn")
        return out if lse is None else (out, lse)


def multicast(allow=None):
    """csa_multicast: let this process's launches use TMA multicast or not (None: leave it); returns what held
    before.  A rank of a job over several GPUs turns it off first."""
    return bool(lib().csa_multicast(-1 if allow is None else int(bool(allow))))


def rmsnorm(x, w, eps, out=None, stream=None):
    N = x.shape[-1]
    out = torch.empty_like(x) if out is None else out
    _check(lib().csa_rmsnorm(_dev(x, torch.bfloat16, "x"), x.numel() // N, N, _dev(w, torch.float32, "w"), eps, _dev(out, torch.bfloat16, "out"),
                             _stream(stream)), "csa_rmsnorm")
    return out


def rope(x, rd, pos, tab, inverse=False, rows_per_pos=1, stream=None):
    """In place on x [rows, row_len]."""
    row_len = x.shape[-1]
    _check(lib().csa_rope(_dev(x, torch.bfloat16, "x"), x.numel() // row_len, row_len, rd, _dev(pos, torch.int32, "pos"), rows_per_pos,
                          _dev(tab, torch.float32, "tab"), tab.shape[0], int(inverse), _stream(stream)), "csa_rope")
    return x


def act_quant(x, codes=None, scale_exp=None, stream=None):
    """In place on x; codes uint8 like x, scale_exp int8 [n/32]."""
    _check(lib().csa_act_quant(_dev(x, torch.bfloat16, "x"), x.numel(), _dev(codes, torch.uint8, "codes"), _dev(scale_exp, torch.int8, "scale_exp"),
                               _stream(stream)), "csa_act_quant")
    return x


def kv_finish(kv_in, kv_out, B, T, start_pos, rd, tab, ring, win_idx=None, codes=None, scales=None, stream=None):
    hd = kv_in.shape[-1]
    W = ring.shape[1]
    _check(lib().csa_kv_finish(_dev(kv_in, torch.bfloat16, "kv_in"), _dev(kv_out, torch.bfloat16, "kv_out"), B, T, start_pos, hd, rd,
                               _dev(tab, torch.float32, "tab"), tab.shape[0], _dev(ring, torch.bfloat16, "ring"), W, _dev(win_idx, torch.int32, "win_idx"),
                               0 if win_idx is None else win_idx.shape[-1], _dev(codes, torch.uint8, "codes"),
                               _dev(scales, torch.int8, "scales"), _stream(stream)), "csa_kv_finish")


def index_scores(qI, wI, KI, B, T, start_pos, compress_len, ratio, S, cand=None, cand_block=1, stream=None):
    n, Hi, dI = qI.shape
    _check(lib().csa_index_scores(_dev(qI, torch.bfloat16, "qI"), _dev(wI, torch.float32, "wI"), _dev(KI, torch.bfloat16, "KI"), B, T, start_pos, Hi, dI,
                                  KI.shape[1], compress_len, ratio, _dev(cand, torch.uint8, "cand"),
                                  0 if cand is None else cand.shape[-1], cand_block, _dev(S, torch.float32, "S"), _stream(stream)),
           "csa_index_scores")
    return S


def candidate_blocks(S, B, T, start_pos, compress_len, ratio, cand_block, K, mask, stream=None):
    """csa_candidate_blocks: mask uint8 [B*T, cand_width] from the scores S f32 [B*T, L]."""
    _check(lib().csa_candidate_blocks(_dev(S, torch.float32, "S"), B, T, start_pos, S.shape[-1], compress_len, ratio,
                                      cand_block, K, _dev(mask, torch.uint8, "mask"), mask.shape[-1], _stream(stream)),
           "csa_candidate_blocks")
    return mask


def index_topk(S, B, T, start_pos, compress_len, ratio, K, out, offset=0, cand=None, cand_block=1, stream=None):
    _check(lib().csa_index_topk(_dev(S, torch.float32, "S"), B, T, start_pos, S.shape[-1], compress_len, ratio,
                                _dev(cand, torch.uint8, "cand"), 0 if cand is None else cand.shape[-1], cand_block, K, offset,
                                _dev(out, torch.int32, "out"), _stream(stream)), "csa_index_topk")
    return out


def page_step(new_len, length, table, free, state, page, tok_req, tok_pos, tok_slot, cu=None, length_out=None,
              state_out=None, info=None, stream=None):
    """csa_page_step: the token maps and tables of one step of a continuous batch.  new_len, length int32 [R]; table
    int32 [R, width]; free int32 [n_pages], state int32 [2] the ring of free pages; tok_req, tok_pos, tok_slot int32
    [N], cu int32 [R+1].  length_out, state_out: where the state after the step goes (default: length and state
    themselves).  Returns info int32 [4]: tokens, pages taken, pages released, error bits."""
    R, N = new_len.numel(), tok_req.numel()
    dev, st = _now(stream)
    if table.dim() != 2 or table.shape[0] != R:
        raise ValueError("table: expected [%d, width], got %s" % (R, tuple(table.shape)))
    if info is None:
        info = _empty((4,), torch.int32, new_len.device, stream)
    i32, width, n_pages = torch.int32, table.shape[1], free.numel()
    lp, sp = _vec(length, R, i32, dev, "length"), _vec(state, 2, i32, dev, "state")
    _check(lib().csa_page_step(
        _vec(new_len, R, i32, dev, "new_len"), R, page, lp, _vec(table, R * width, i32, dev, "table"), width,
        _vec(free, n_pages, i32, dev, "free"), n_pages, sp, _vec(tok_req, N, i32, dev, "tok_req"),
        _vec(tok_pos, N, i32, dev, "tok_pos"), _vec(tok_slot, N, i32, dev, "tok_slot"), N, _vec(cu, R + 1, i32, dev, "cu"),
        lp if length_out is None else _vec(length_out, R, i32, dev, "length_out"),
        sp if state_out is None else _vec(state_out, 2, i32, dev, "state_out"), _vec(info, 4, i32, dev, "info"), st),
        "csa_page_step")
    return info
