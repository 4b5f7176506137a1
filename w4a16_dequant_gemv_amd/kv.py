"""torch-facing wrappers over the KV-cache codec of libw4a16.so
(`include/kv_codec.h`): V quantized per token, K per channel over blocks of
tokens, symmetric INT8 or INT4 codes in int8, fp32 scales; and the paged INT8
cache (PagedKVCache): appending new tokens with rotation, and attention over it.

Only argument marshalling happens here: tensors must already live on the GPU
and the library does all of the arithmetic on torch's current stream.
"""
from ctypes import byref, create_string_buffer
from functools import lru_cache

import torch

from . import _lib
from ._lib import W4A16Error, check, lib
from .api import _need, _raw_stream, _same_device, _stream


def _dev_tensor(t, dtype, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise W4A16Error(f"{name} must be a GPU tensor (there is no CPU implementation)")
    if t.dtype != dtype:
        raise W4A16Error(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise W4A16Error(f"{name} must be contiguous")


def quant_tokens(x, bits=8, q=None, scale=None):
    """fp16 x [..., d] -> (int8 q [..., d], fp32 scale [...]): one symmetric
    scale per token row over the head dimension (the V side)."""
    _dev_tensor(x, torch.float16, "x")
    d = x.shape[-1]
    rows = x.numel() // d
    q = torch.empty(x.shape, dtype=torch.int8, device=x.device) if q is None else q
    scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device) if scale is None else scale
    _need(q, torch.int8, x.shape, "q")
    _need(scale, torch.float32, x.shape[:-1], "scale")
    _same_device(x, q, scale)
    with torch.cuda.device(x.device):
        check(lib().kv_quant_tokens(x.data_ptr(), rows, d, bits, q.data_ptr(), scale.data_ptr(), _stream(x)),
              "kv_quant_tokens")
    return q, scale


def quant_channels(x, bits=8, q=None, scale=None):
    """fp16 x [blocks, t, d] -> (int8 q [blocks, t, d], fp32 scale [blocks, d]):
    one symmetric scale per channel of each block of t tokens (the K side)."""
    _dev_tensor(x, torch.float16, "x")
    if x.dim() != 3:
        raise W4A16Error("x must be [blocks, t, d]")
    blocks, t, d = x.shape
    q = torch.empty(x.shape, dtype=torch.int8, device=x.device) if q is None else q
    scale = torch.empty((blocks, d), dtype=torch.float32, device=x.device) if scale is None else scale
    _need(q, torch.int8, x.shape, "q")
    _need(scale, torch.float32, (blocks, d), "scale")
    _same_device(x, q, scale)
    with torch.cuda.device(x.device):
        check(lib().kv_quant_channels(x.data_ptr(), blocks, t, d, bits, q.data_ptr(), scale.data_ptr(),
                                      _stream(x)), "kv_quant_channels")
    return q, scale


def dequant_tokens(q, scale, out=None):
    """int8 q [..., d], fp32 scale [...] -> fp16 q * scale."""
    _dev_tensor(q, torch.int8, "q")
    d = q.shape[-1]
    _need(scale, torch.float32, q.shape[:-1], "scale")
    out = torch.empty(q.shape, dtype=torch.float16, device=q.device) if out is None else out
    _need(out, torch.float16, q.shape, "out")
    _same_device(q, scale, out)
    with torch.cuda.device(q.device):
        check(lib().kv_dequant_tokens(q.data_ptr(), scale.data_ptr(), q.numel() // d, d, out.data_ptr(),
                                      _stream(q)), "kv_dequant_tokens")
    return out


def dequant_channels(q, scale, out=None):
    """int8 q [blocks, t, d], fp32 scale [blocks, d] -> fp16 q * scale."""
    _dev_tensor(q, torch.int8, "q")
    if q.dim() != 3:
        raise W4A16Error("q must be [blocks, t, d]")
    blocks, t, d = q.shape
    _need(scale, torch.float32, (blocks, d), "scale")
    out = torch.empty(q.shape, dtype=torch.float16, device=q.device) if out is None else out
    _need(out, torch.float16, q.shape, "out")
    _same_device(q, scale, out)
    with torch.cuda.device(q.device):
        check(lib().kv_dequant_channels(q.data_ptr(), scale.data_ptr(), blocks, t, d, out.data_ptr(),
                                        _stream(q)), "kv_dequant_channels")
    return out


class KVBlockPool:
    """A pool of quantized KV blocks of t tokens x d channels for one layer's
    heads: K codes with per-channel scales, V codes with per-token scales."""

    def __init__(self, pool_blocks, t, d, device, bits=8):
        self.t, self.d, self.bits = t, d, bits
        self.k = torch.zeros((pool_blocks, t, d), dtype=torch.int8, device=device)
        self.k_scale = torch.zeros((pool_blocks, d), dtype=torch.float32, device=device)
        self.v = torch.zeros((pool_blocks, t, d), dtype=torch.int8, device=device)
        self.v_scale = torch.zeros((pool_blocks, t), dtype=torch.float32, device=device)

    @property
    def pool_blocks(self):
        return self.k.shape[0]

    def flush(self, k_blocks, v_blocks, dst):
        """Quantize fp16 window blocks k_blocks / v_blocks [P, t, d] into the
        slots dst (int32 [P] on the GPU); slots outside the pool are skipped."""
        for name, tns in (("k_blocks", k_blocks), ("v_blocks", v_blocks)):
            _dev_tensor(tns, torch.float16, name)
        P = k_blocks.shape[0]
        _need(v_blocks, torch.float16, (P, self.t, self.d), "v_blocks")
        _need(k_blocks, torch.float16, (P, self.t, self.d), "k_blocks")
        _need(dst, torch.int32, (P,), "dst")
        _same_device(k_blocks, v_blocks, dst, self.k)
        with torch.cuda.device(self.k.device):
            check(lib().kv_flush_blocks(k_blocks.data_ptr(), v_blocks.data_ptr(), P, self.t, self.d, self.bits,
                                        dst.data_ptr(), self.pool_blocks, self.k.data_ptr(),
                                        self.k_scale.data_ptr(), self.v.data_ptr(), self.v_scale.data_ptr(),
                                        _stream(self.k)), "kv_flush_blocks")


def rope_table(rows, dim, base=10000.0, device="cuda"):
    """Cosine and sine of position p times base^(-2 j / dim), fp32 [rows, dim/2, 2]
    (angles in binary64: positions lose whole turns in binary32)."""
    f = float(base) ** (-torch.arange(0, dim, 2, dtype=torch.float64, device=device) / dim)
    a = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * f
    return torch.stack((a.cos(), a.sin()), -1).float()


def _fits(t, dtype, shape, device, name):
    """Raise unless t is a contiguous GPU tensor of this dtype and shape on `device`."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous()):
        _need(t, dtype, shape, name)
        raise W4A16Error("all tensors must be on the same GPU")


def _heads(t, heads, d, name, device):
    """The row stride of fp16 t [T, heads, d] whose rows are whole (a view into
    a fused projection's output is)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise W4A16Error(f"{name} must be a GPU tensor (there is no CPU implementation)")
    shape = t.shape
    if t.dtype is not torch.float16 or len(shape) != 3 or shape[2] != d or (heads is not None and shape[1] != heads):
        raise W4A16Error(f"{name} must be float16 [tokens, {'heads' if heads is None else heads}, {d}], got "
                         f"{t.dtype} {tuple(shape)}")
    if t.device != device:
        raise W4A16Error("all tensors must be on the same GPU")
    row, head, one = t.stride()
    if one != 1 or (head != d and shape[1] > 1):
        raise W4A16Error(f"{name}: a token's heads must lie side by side")
    return row if shape[0] > 1 else shape[1] * d


@lru_cache(maxsize=4096)
def _workspace_size(tokens, batch, n_q, n_kv, d):
    """By these sizes alone, so asked once for each (0.7 us of a call on the host)."""
    return lib().kv_paged_attention_workspace_size(tokens, batch, n_q, n_kv, d)


@lru_cache(maxsize=4096)
def _shared_workspace_size(*sizes):
    return lib().kv_paged_attention_shared_workspace_size(*sizes)


def attention_config(tokens, batch, table_cols, n_q, n_kv, d, page=128, window=0, sinks=0, groups=0, max_pages=0):
    """Names of the kernels that PagedKVCache.attend launches for `tokens` queries of
    `batch` sequences with block tables of `table_cols` pages (with `groups` and
    `max_pages` of a SharedPrefix), as profilers print them.  Nothing is launched; works
    without a GPU."""
    name = create_string_buffer(256)
    if groups:
        if window or sinks:
            raise W4A16Error("a shared prefix takes no window")
        check(lib().kv_paged_attention_shared_config(tokens, batch, table_cols, page, groups, max_pages, n_q, n_kv, d,
                                                     name, len(name)), "kv_paged_attention_shared_config")
        return name.value.decode()
    check(lib().kv_paged_attention_config(tokens, batch, table_cols, page, n_q, n_kv, d, window, sinks, name, len(name)),
          "kv_paged_attention_config")
    return name.value.decode()


class _Kept:
    """Copies and pickles go without the library's struct, whose addresses are not theirs."""

    _known = None                    # what the last check found, and the struct for it

    def __getstate__(self):
        return {**self.__dict__, "_known": None}


class PagedBatch(_Kept):
    """The sequences of one call (kv_paged_batch in kv_codec.h), int32 GPU
    tensors: rows cu_q[b] .. cu_q[b+1]-1 of the call belong to sequence b, which
    holds ctx_lens[b] tokens before them; its page p is pool page
    block_table[b, p], its ring of fp16 pages is slots[b].  The tensors are read
    when the kernels run, so one PagedBatch can be kept (and captured) while
    their contents change from step to step."""

    def __init__(self, cu_q, ctx_lens, block_table, slots):
        if not isinstance(ctx_lens, torch.Tensor) or not isinstance(block_table, torch.Tensor):
            raise W4A16Error("ctx_lens and block_table must be GPU tensors")
        if ctx_lens.dim() != 1 or block_table.dim() != 2 or ctx_lens.numel() == 0 or block_table.shape[1] == 0:
            raise W4A16Error("ctx_lens must be [batch], block_table [batch, pages per sequence], neither empty")
        B = ctx_lens.shape[0]
        for t, shape, name in ((cu_q, (B + 1,), "cu_q"), (ctx_lens, (B,), "ctx_lens"),
                               (block_table, (B, block_table.shape[1]), "block_table"), (slots, (B,), "slots")):
            _need(t, torch.int32, shape, name)
        _same_device(cu_q, ctx_lens, block_table, slots)
        self._tensors, self._device = (cu_q, ctx_lens, block_table, slots), cu_q.device
        self._known, self._sizes = None, (*(t.numel() for t in self._tensors), block_table.shape[1])

    cu_q = property(lambda self: self._tensors[0])
    ctx_lens = property(lambda self: self._tensors[1])
    block_table = property(lambda self: self._tensors[2])
    slots = property(lambda self: self._tensors[3])

    def _struct(self, tokens, device):
        """The library's struct for a call of so many tokens, and the number of sequences."""
        if self._device != device:
            raise W4A16Error("all tensors must be on the same GPU")
        q, c, t, s = self._tensors
        if (q.numel(), c.numel(), t.numel(), s.numel(), t.shape[-1]) != self._sizes or not t.is_contiguous():
            self.__init__(q, c, t, s)                          # changed in place: checked again
        at = (q.data_ptr(), c.data_ptr(), t.data_ptr(), s.data_ptr(), tokens)
        known = self._known
        if known is None or known[0] != at:
            B = c.shape[0]
            known = self._known = at, (byref(_lib.PagedBatch(*at, B, t.shape[1])), B)
        return known[1]


class SharedPrefix(_Kept):
    """Groups of a batch's sequences that begin with the same tokens (kv_shared_prefix in
    kv_codec.h), int32 GPU tensors: sequences cu_seqs[g] .. cu_seqs[g+1]-1 have the same pool
    pages in the first pages[g] columns of their block tables.  max_pages: no group
    shares more (of a group that does, the first max_pages are taken together).  The tensors
    are read when the kernels run, as a PagedBatch's are."""

    def __init__(self, cu_seqs, pages, max_pages):
        if not isinstance(pages, torch.Tensor) or pages.dim() != 1 or not 1 <= pages.shape[0] <= 65536:
            raise W4A16Error("pages must be an int32 GPU tensor [groups] of 1 to 65536 groups")
        G = pages.shape[0]
        _need(cu_seqs, torch.int32, (G + 1,), "cu_seqs")
        _need(pages, torch.int32, (G,), "pages")
        _same_device(cu_seqs, pages)
        if not 1 <= max_pages <= 1 << 24:
            raise W4A16Error(f"max_pages must be in [1, 2^24], got {max_pages}")
        self._tensors, self._device, self._known = (cu_seqs, pages), cu_seqs.device, None
        self._max_pages = int(max_pages)

    cu_seqs = property(lambda self: self._tensors[0])
    pages = property(lambda self: self._tensors[1])
    max_pages = property(lambda self: self._max_pages)

    def _struct(self, device):
        """The library's struct, the number of groups and max_pages."""
        if self._device != device:
            raise W4A16Error("all tensors must be on the same GPU")
        c, p = self._tensors
        if c.numel() != p.numel() + 1 or not (c.is_contiguous() and p.is_contiguous()):
            self.__init__(c, p, self._max_pages)               # changed in place: checked again
        at = (c.data_ptr(), p.data_ptr(), p.numel(), self._max_pages)
        known = self._known
        if known is None or known[0] != at:
            known = self._known = at, (byref(_lib.SharedPrefix(*at)), *at[2:])
        return known[1]


class PagedKVCache(_Kept):
    """One layer's paged INT8 cache (kv_paged_* in kv_codec.h): pages of `page`
    tokens with one scale per (page, kv head) for K and one for V, and a ring of
    the two highest pages that each sequence has reached in fp16, from which the
    unfinished page is read.  Tokens can be taken back to the first one of those
    pages, and beyond that only to a multiple of `page`.  Pages and rings are in
    the order of kv_codec.h; `read` gives pages in the order of tokens.  Block
    tables, lengths and slots are the caller's (PagedBatch), shared by a model's
    layers."""

    def __init__(self, pool_pages, n_kv, d, slots, device, page=128):
        if page not in (64, 128, 256) or d not in (64, 96, 128, 256):
            raise W4A16Error(f"page must be 64, 128 or 256 and d 64, 96, 128 or 256, got {page} and {d}")
        if pool_pages < 1 or slots < 1 or not 1 <= n_kv <= 1024:
            raise W4A16Error("pool_pages and slots must be positive, n_kv in [1, 1024]")
        self.n_kv, self.d, self.page = n_kv, d, page
        kshape, vshape = self._shapes()
        self.k = torch.zeros((pool_pages, *kshape), dtype=torch.int8, device=device)
        self.v = torch.zeros((pool_pages, *vshape), dtype=torch.int8, device=device)
        self.k_scale = torch.zeros((pool_pages, n_kv), dtype=torch.float32, device=device)
        self.v_scale = torch.zeros((pool_pages, n_kv), dtype=torch.float32, device=device)
        self.k_tail = torch.zeros((slots, 2, *kshape), dtype=torch.float16, device=device)
        self.v_tail = torch.zeros((slots, 2, *vshape), dtype=torch.float16, device=device)

    def __setattr__(self, name, value):
        """A replaced tensor is checked by the next call, and let go at once."""
        object.__setattr__(self, "_known", None)
        object.__setattr__(self, name, value)

    def _shapes(self):
        h, d, t = self.n_kv, self.d, self.page
        return (h, t // 64, 4, d // 16, 16, 16), (h, t // 16, d, 16)

    @property
    def pool_pages(self):
        return self.k.shape[0]

    @property
    def slots(self):
        return self.k_tail.shape[0]

    def _checked(self):
        """The six tensors as the library's struct, checked when one was replaced, the
        GPU they are on and its index."""
        k, v, ks, vs, kt, vt = self.k, self.v, self.k_scale, self.v_scale, self.k_tail, self.v_tail
        at = (k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), kt.data_ptr(), vt.data_ptr(),
              k.numel(), v.numel(), ks.numel(), vs.numel(), kt.numel(), vt.numel())
        known = self._known
        if known is not None and known[0] == at:
            return known[1]
        kshape, vshape = self._shapes()
        P, S = self.pool_pages, self.slots
        _need(self.k, torch.int8, (P, *kshape), "k")
        _need(self.v, torch.int8, (P, *vshape), "v")
        _need(self.k_scale, torch.float32, (P, self.n_kv), "k_scale")
        _need(self.v_scale, torch.float32, (P, self.n_kv), "v_scale")
        _need(self.k_tail, torch.float16, (S, 2, *kshape), "k_tail")
        _need(self.v_tail, torch.float16, (S, 2, *vshape), "v_tail")
        _same_device(self.k, self.v, self.k_scale, self.v_scale, self.k_tail, self.v_tail)
        dev = k.device
        known = self._known = at, (byref(_lib.PagedCache(*at[:6], P, S, self.n_kv, self.d, self.page)), dev, dev.index)
        return known[1]

    def append(self, k, v, batch, q=None, rope=None, positions=None, interleaved=False, q_out=None):
        """Put fp16 k, v [T, n_kv, d] behind each sequence's ctx_lens tokens; with
        `rope` (fp32 [rows, dim/2, 2], see rope_table) and int32 positions [T], k
        is rotated first, and q [T, n_q, d] into the result [T, n_q, d] (None
        without q).  ctx_lens is not changed: advance it once every layer has
        appended and attended."""
        c, dev, gpu = self._checked()
        ks, vs = _heads(k, self.n_kv, self.d, "k", dev), _heads(v, self.n_kv, self.d, "v", dev)
        T = k.shape[0]
        if v.shape[0] != T:
            raise W4A16Error("k and v must have the same tokens")
        if rope is None:
            if q is not None or positions is not None:
                raise W4A16Error("q and positions are only used with rope")
            if T:
                self._call("kv_paged_append", gpu, c, batch._struct(T, dev)[0], k.data_ptr(), ks, v.data_ptr(), vs,
                           None, 0, 0, None, 0, 0, 0, None, None)
            return None
        if not isinstance(rope, torch.Tensor) or rope.dim() != 3:
            raise W4A16Error("rope must be fp32 [rows, dim/2, 2] on the GPU")
        rows, pairs, _ = rope.shape
        _fits(rope, torch.float32, (rows, pairs, 2), dev, "rope")
        if rows < 1 or pairs < 16 or pairs % 16 or pairs * 2 > self.d:
            raise W4A16Error(f"rope must rotate a multiple of 32 channels, at most d={self.d}")
        _fits(positions, torch.int32, (T,), dev, "positions")
        qs = n_q = q_at = out_at = None
        if q is not None:
            qs, n_q = _heads(q, None, self.d, "q", dev), q.shape[1]
            if q.shape[0] != T:
                raise W4A16Error("q and k must have the same tokens")
            if q_out is None:
                q_out = q.new_empty((T, n_q, self.d))
            else:
                _fits(q_out, torch.float16, (T, n_q, self.d), dev, "q_out")
            q_at, out_at = q.data_ptr(), q_out.data_ptr()
        if T:
            self._call("kv_paged_append", gpu, c, batch._struct(T, dev)[0], k.data_ptr(), ks, v.data_ptr(), vs,
                       q_at, qs or 0, n_q or 0, rope.data_ptr(), rows, pairs * 2, 1 if interleaved else 0,
                       positions.data_ptr(), out_at)
        return None if q is None else q_out

    @staticmethod
    def _call(name, gpu, *args):
        """A library call on torch's current stream of that GPU, made the current one."""
        fn = getattr(lib(), name)
        stream = _raw_stream(gpu)
        if torch.cuda.current_device() == gpu:
            rc = fn(*args, stream)
        else:
            with torch.cuda.device(gpu):
                rc = fn(*args, stream)
        if rc:
            check(rc, name)

    def read(self, ids, k_out=None, v_out=None):
        """Pool pages ids (int32 [n]) as fp16 (K, V), each [n, n_kv, page, d] in the
        order of tokens; ids outside the pool are skipped."""
        c, dev, gpu = self._checked()
        if not isinstance(ids, torch.Tensor) or ids.dim() != 1:
            raise W4A16Error("ids must be int32 [n] on the GPU")
        n = ids.shape[0]
        _fits(ids, torch.int32, (n,), dev, "ids")
        shape = (n, self.n_kv, self.page, self.d)
        if k_out is None:
            k_out = self.k_tail.new_empty(shape)
        else:
            _fits(k_out, torch.float16, shape, dev, "k_out")
        if v_out is None:
            v_out = self.k_tail.new_empty(shape)
        else:
            _fits(v_out, torch.float16, shape, dev, "v_out")
        if n:
            self._call("kv_paged_read", gpu, c, ids.data_ptr(), n, k_out.data_ptr(), v_out.data_ptr())
        return k_out, v_out

    def attend(self, q, batch, scale=None, window=0, sinks=0, out=None, workspace=None, prefix=None):
        """softmax(scale * q k^T) v of fp16 q [T, n_q, d] over the cache, into fp16
        [T, n_q, d]; the batch's own tokens have been appended before.  Row i of
        a sequence sees the tokens up to its own, with window > 0 the last
        `window` of them and the sequence's first `sinks`.  scale defaults to
        d^-1/2.  Rows of no sequence are left as they were.  With `prefix` (a
        SharedPrefix; no window) the pages that a group of sequences share are read and
        scored once for all of its rows: the same result but for the order of sums.  Calls of
        more than 64 rows a kv head for each sequence on average are run as without one, so
        a long chunk of a prompt is better called apart from the others' single tokens."""
        c, dev, gpu = self._checked()
        qs = _heads(q, None, self.d, "q", dev)
        T, n_q = q.shape[:2]
        if n_q == 0 or n_q % self.n_kv or n_q > 1024:
            raise W4A16Error(f"q must have a multiple of {self.n_kv} heads, at most 1024, got {n_q}")
        if window < 0 or sinks < 0 or (sinks and not window) or max(window, sinks) >= 1 << 31:
            raise W4A16Error("window and sinks must not be negative, and sinks need a window")
        if window and prefix is not None:
            raise W4A16Error("a shared prefix takes no window")
        scale = self.d ** -0.5 if scale is None else float(scale)
        if not 0.0 < scale <= 1e6:
            raise W4A16Error(f"scale must be in (0, 1e6], got {scale}")
        if out is None:
            out = q.new_empty((T, n_q, self.d))
        else:
            _fits(out, torch.float16, (T, n_q, self.d), dev, "out")
        if T == 0:
            return out
        b, B = batch._struct(T, dev)
        if prefix is None:
            need = _workspace_size(T, B, n_q, self.n_kv, self.d)
        elif not isinstance(prefix, SharedPrefix):
            raise W4A16Error("prefix must be a SharedPrefix")
        else:
            p, groups, max_pages = prefix._struct(dev)
            need = _shared_workspace_size(T, B, batch.block_table.shape[1], self.page, groups, max_pages, n_q, self.n_kv, self.d)
        if workspace is None:
            workspace = self.k.new_empty(need)
        elif not isinstance(workspace, torch.Tensor) or workspace.device != dev or not workspace.is_contiguous():
            raise W4A16Error("workspace must be a contiguous tensor on the cache's GPU")
        at, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        if prefix is None:
            self._call("kv_paged_attention", gpu, c, b, q.data_ptr(), qs, n_q, scale, window, sinks, at, size,
                       out.data_ptr())
        else:
            self._call("kv_paged_attention_shared", gpu, c, b, p, q.data_ptr(), qs, n_q, scale, at, size, out.data_ptr())
        return out
