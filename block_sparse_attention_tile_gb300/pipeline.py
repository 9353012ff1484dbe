"""The hot path end to end, composed from the C-ABI entry points.

Each function allocates the outputs and intermediates with torch (device
memory is the only thing torch provides here) and calls the library's
stages in order on the current stream.  No arithmetic of the method happens
in Python.
"""

import math
from dataclasses import dataclass
from typing import NamedTuple, Optional

import torch

from . import bsa


@dataclass
class Geometry:
    """Token layout of one sequence: an optional dense prefix of ``n_prefix``
    tokens, then a (T, H, W) video grid cut into (bT, bH, bW) blocks, or, when
    ``perm`` is given, into runs of M consecutive entries of that permutation
    of the raster video order.  M is the block capacity."""
    T: int
    H: int
    W: int
    bT: int = 1
    bH: int = 1
    bW: int = 1
    M: int = 128
    n_prefix: int = 0
    perm: Optional[torch.Tensor] = None  # int32 [T*H*W] on the device

    @property
    def n_tokens(self):
        return self.n_prefix + self.T * self.H * self.W

    @property
    def prefix_blocks(self):
        return -(-self.n_prefix // self.M)

    @property
    def geometry(self):
        """The tiling as the 8 host integers the attention entry points take."""
        return [self.T, self.H, self.W, self.bT, self.bH, self.bW, self.n_prefix, 1 if self.perm is not None else 0]

    @property
    def num_blocks(self):
        return bsa.bsa_tile_count(self.T, self.H, self.W, self.bT, self.bH, self.bW, self.n_prefix,
                                  self.perm is not None, self.M)


@dataclass
class SegmentGeometry:
    """An ordered list of segments (an int: a dense segment of that many
    tokens, e.g. text, image or audio; a (T, H, W) tuple: a video grid, e.g. a
    reference video or the target video), token ids counting along that
    order.  Dense segments are chunked first, the videos follow in order, each
    in (bT, bH, bW) windows with its own block span (the routing regions)."""
    segments: list
    bT: int = 1
    bH: int = 1
    bW: int = 1
    M: int = 128
    perm = None
    geometry = None  # no single video grid: the attention reads tiles by index

    def __post_init__(self):
        self.segments = [s if isinstance(s, int) else tuple(s) for s in self.segments]
        self._J, self._P, self._spans = bsa.bsa_segments_count(self.segments, self.bT, self.bH, self.bW, self.M)

    @property
    def n_tokens(self):
        return sum(s if isinstance(s, int) else s[0] * s[1] * s[2] for s in self.segments)

    @property
    def num_blocks(self):
        return self._J

    @property
    def prefix_blocks(self):
        return self._P

    @property
    def spans(self):
        """Block range [lo, hi) of each video segment, in tiled order."""
        return list(self._spans)


def tile_map(geom, device="cuda"):
    J = geom.num_blocks
    index_map = torch.empty((J, geom.M), dtype=torch.int32, device=device)
    block_sizes = torch.empty((J,), dtype=torch.int32, device=device)
    if isinstance(geom, SegmentGeometry):
        bsa.bsa_tile_map_segments(geom.segments, geom.bT, geom.bH, geom.bW, geom.M, index_map, block_sizes)
    else:
        bsa.bsa_tile_map(geom.T, geom.H, geom.W, geom.bT, geom.bH, geom.bW, geom.n_prefix, geom.perm, geom.M,
                         index_map, block_sizes)
    return index_map, block_sizes


@dataclass
class BlockSparseResult:
    out: torch.Tensor
    lse: Optional[torch.Tensor]
    index_map: torch.Tensor
    block_sizes: torch.Tensor
    qbar: torch.Tensor
    kbar: torch.Tensor
    q2k_idx: torch.Tensor
    q2k_num: torch.Tensor
    packed: Optional[torch.Tensor] = None
    summary_bias: Optional[torch.Tensor] = None
    coarse: Optional[torch.Tensor] = None


def block_sparse_attention(q, k, v, geom, topk, scale=None, kmax=None, summary=False, need_lse=True,
                           tiles=None, pass_geometry=True, packed=None, reweight=False, coarse_gate=None):
    """Tile map -> pool -> route -> block-sparse (or exact+summary) attention.

    q, k, v: [BH, N, D] (BHSD) float32 or bfloat16 on the device.  Routing
    covers the video blocks; prefix blocks are always attended.  With a
    SegmentGeometry, ``topk`` may be a list with one budget per video segment:
    the region-grouped TopK keeps that many blocks of each segment per row.  ``packed``:
    let the pool pass also write Q/K/V in block order for the attention to
    read (default: when the blocks come from a permutation, whose rows the
    tensor-core kernel would otherwise gather four at a time).  Returns the
    output in raster order plus every intermediate.  ``reweight`` (with
    ``summary``): the unselected blocks are summarised by Spark-Reweight
    (weighted key and value at the head's mean video query, log-mass bias)
    instead of by their means and log(n_j).  ``coarse_gate`` (float32 [BH, D]
    per head and channel, or [BH, N, D] per token): add the gated coarse
    branch softmax(E) V_bar of each routed query block to its tokens."""
    BH, N, D = q.shape
    assert N == geom.n_tokens
    dev = q.device
    scale = D ** -0.5 if scale is None else scale
    index_map, block_sizes = tile_map(geom, dev) if tiles is None else tiles
    J = index_map.shape[0]
    P = geom.prefix_blocks
    Jr = J - P
    grouped = not isinstance(topk, int)
    if grouped:
        spans = geom.spans
        assert len(topk) == len(spans), "one budget per video segment"
        kept = sum(min(kr, hi - lo) for kr, (lo, hi) in zip(topk, spans))
        kmax = kept if kmax is None else kmax
    else:
        kmax = topk if kmax is None else kmax
    if packed is None:
        # tiles that are not one box of a single video grid: gather them once in the pool pass
        packed = ((geom.perm is not None or isinstance(geom, SegmentGeometry)) and q.dtype == torch.bfloat16
                  and D == 128 and geom.M == 128)
    pk = torch.empty((3, BH, J, geom.M, D), dtype=q.dtype, device=dev) if packed else None
    qbar = torch.empty((BH, J, D), dtype=torch.float32, device=dev)
    kbar = torch.empty_like(qbar)
    coarse = coarse_gate is not None
    vbar = torch.empty_like(qbar) if (summary or packed or coarse) else None
    kbar_lp = torch.empty((BH, J, D), dtype=q.dtype, device=dev) if summary else None
    vbar_lp = torch.empty((BH, J, D), dtype=q.dtype, device=dev) if summary else None
    bsa.bsa_pool_blocks(q, k, v if vbar is not None else None, BH, N, D, index_map, block_sizes, J, geom.M,
                        qbar, kbar, vbar, kbar_lp, vbar_lp, packed=pk)
    q2k_idx = torch.empty((BH, Jr, kmax), dtype=torch.int32, device=dev)
    q2k_num = torch.empty((BH, Jr), dtype=torch.int32, device=dev)
    ws = torch.empty((bsa.bsa_route_workspace(BH, Jr) // 4,), dtype=torch.float32, device=dev)
    if grouped:
        starts = [lo - P for lo, _ in geom.spans] + [Jr]
        bsa.bsa_route_topk_grouped(qbar[:, P:], kbar[:, P:], BH, Jr, D, J * D, starts, list(topk), scale, kmax,
                                   q2k_idx, q2k_num, ws)
    else:
        bsa.bsa_route_topk(qbar[:, P:], kbar[:, P:], BH, Jr, D, J * D, topk, scale, kmax, q2k_idx, q2k_num, ws)
    sbias = None
    if summary and reweight:
        sbias = torch.empty((BH, J), dtype=torch.float32, device=dev)
        rws = torch.empty((bsa.bsa_reweight_workspace(BH, D) // 4,), dtype=torch.float32, device=dev)
        bsa.bsa_reweight_summaries(q, k, v, BH, N, D, index_map, block_sizes, J, geom.M, P, scale, kbar_lp, vbar_lp,
                                   sbias, rws, qbar=qbar, packed=pk)
    out = torch.empty_like(q)
    lse = torch.empty((BH, N), dtype=torch.float32, device=dev) if need_lse else None
    if summary:
        bsa.bsa_fwd_summary(q, k, v, BH, N, D, index_map, block_sizes, J, geom.M, P, geom.geometry if pass_geometry else None,
                            q2k_idx, q2k_num, kmax, kbar_lp, vbar_lp, scale, out, lse, packed=pk, summary_bias=sbias)
    else:
        bsa.bsa_fwd_qouter(q, k, v, BH, N, D, index_map, block_sizes, J, geom.M, P, geom.geometry if pass_geometry else None,
                           q2k_idx, q2k_num, kmax, scale, out, lse, packed=pk)
    C = None
    if coarse:
        # E is the route's own score matrix, left in its workspace
        C = torch.empty((BH, Jr, D), dtype=torch.float32, device=dev)
        bsa.bsa_coarse_attention(ws, Jr * Jr, vbar[:, P:], J * D, BH, Jr, D, C)
        bsa.bsa_coarse_apply(out, C, coarse_gate, coarse_gate.dim() == 3, BH, N, D, index_map, block_sizes, J,
                             geom.M, P)
    return BlockSparseResult(out, lse, index_map, block_sizes, qbar, kbar, q2k_idx, q2k_num, pk, sbias, C)


@dataclass
class ReblockedResult:
    out: torch.Tensor
    lse: Optional[torch.Tensor]
    perm: torch.Tensor              # [BH, N - n_prefix] the layout of each head
    inner: BlockSparseResult        # the attention in the layout's order


def reblocked_attention(q, k, v, n_prefix, M, topk, scale=None, summary=False, reweight=False, need_lse=True,
                        ridge=1e-6):
    """Spark-Reblock layout -> rows gathered into it -> the block-sparse path
    over consecutive runs of M -> outputs scattered back to the original
    order.  q, k, v: [BH, N, D] with a dense prefix of n_prefix tokens (always
    attended, not reblocked) followed by the video tokens."""
    BH, N, D = q.shape
    Nv = N - n_prefix
    dev = q.device
    perm = torch.empty((BH, Nv), dtype=torch.int32, device=dev)
    ws = torch.empty((bsa.bsa_reblock_workspace(BH, N, D, n_prefix),), dtype=torch.uint8, device=dev)
    bsa.bsa_reblock_layout(q, k, BH, N, D, n_prefix, M, perm, ws, ridge=ridge)
    q2, k2, v2 = (torch.empty_like(x) for x in (q, k, v))
    for src, dst in ((q, q2), (k, k2), (v, v2)):
        bsa.bsa_permute_rows(src, dst, BH, N, D, n_prefix, perm)
    # in the layout's order every block is a run of M consecutive rows: a (1, 1, Nv) grid in (1, 1, M) windows
    geom = Geometry(1, 1, Nv, 1, 1, M, M=M, n_prefix=n_prefix)
    inner = block_sparse_attention(q2, k2, v2, geom, topk, scale=scale, summary=summary, reweight=reweight,
                                   need_lse=need_lse)
    out = torch.empty_like(q)
    bsa.bsa_permute_rows(inner.out, out, BH, N, D, n_prefix, perm, inverse=True)
    lse = None
    if need_lse:
        lse = torch.empty_like(inner.lse)
        bsa.bsa_permute_rows(inner.lse.view(BH, N, 1), lse.view(BH, N, 1), BH, N, 1, n_prefix, perm, inverse=True)
    return ReblockedResult(out, lse, perm, inner)


def nsa_qouter(q, k, v, block_indices, block_counts, block_size, causal=True, scale=None, need_lse=True):
    """Token-granular GQA selected attention, query-outer.  q [B,T,HQ,D],
    k/v [B,T,H,D], block_indices [B,T,H,S] int32, block_counts [B,T,H] int32."""
    B, T, HQ, D = q.shape
    H = k.shape[2]
    S = block_indices.shape[-1]
    scale = D ** -0.5 if scale is None else scale
    out = torch.empty_like(q)
    lse = torch.empty((B, T, HQ), dtype=torch.float32, device=q.device) if need_lse else None
    bsa.bsa_fwd_qouter_tokens(q, k, v, B, T, HQ, H, D, block_indices, block_counts, S, block_size, causal,
                              scale, out, lse)
    return out, lse


@dataclass
class KVOuterPlan:
    row_ptr: torch.Tensor
    q_idx: torch.Tensor
    slot: torch.Tensor
    chunks: torch.Tensor
    n_chunks: torch.Tensor
    max_chunks: int
    nblk: int
    window: int = 0


# Query positions per window of the KV-outer order (0: one window).  Windows
# make the grid work through one window of queries at a time, so each query row
# is read from HBM once (measured: 58% fewer DRAM reads in the partial pass at
# the MSA shape), but they add K/V segments; the partial pass is bound by its
# softmax -> P V -> epilogue chain, not by HBM, so the default is one window.
KV_WINDOW = 0


def default_window(N):
    return KV_WINDOW if 0 < KV_WINDOW < N else 0


def windows(N, window):
    return 1 if window <= 0 or window >= N else -(-N // window)


def reverse_index(block_indices, block_counts, nblk, chunk_cap, workspace=None, window=None):
    B, N, H, S = block_indices.shape
    dev = block_indices.device
    window = default_window(N) if window is None else window
    max_chunks = bsa.bsa_max_chunks(B, N, H, S, nblk, chunk_cap, window)
    row_ptr = torch.empty((B * windows(N, window) * H * nblk + 1,), dtype=torch.int32, device=dev)
    q_idx = torch.empty((B * H * N * S,), dtype=torch.int32, device=dev)
    slot = torch.empty_like(q_idx)
    chunks = torch.empty((max_chunks, 4), dtype=torch.int32, device=dev)
    n_chunks = torch.empty((1,), dtype=torch.int32, device=dev)
    if workspace is None:
        ws = bsa.bsa_reverse_index_workspace(B, N, H, nblk)
        workspace = torch.empty((max(ws, 16),), dtype=torch.uint8, device=dev)
    bsa.bsa_build_reverse_index(block_indices, block_counts, B, N, H, S, nblk, chunk_cap, row_ptr, q_idx,
                                slot, chunks, n_chunks, max_chunks, workspace, window=window)
    return KVOuterPlan(row_ptr, q_idx, slot, chunks, n_chunks, max_chunks, nblk, window)


def kvouter_attention(q, k, v, block_indices, block_counts, block_size, causal=True, scale=None,
                      chunk_cap=None, obuf_dtype=torch.bfloat16, need_lse=True, plan=None, window=None):
    """KV-outer order: reverse index -> partial pass -> combine.  Same inputs
    and result as nsa_qouter."""
    B, N, HQ, D = q.shape
    H = k.shape[2]
    S = block_indices.shape[-1]
    scale = D ** -0.5 if scale is None else scale
    nblk = -(-N // block_size)
    if chunk_cap is None:
        chunk_cap = 2 * S * block_size
    if plan is None:
        plan = reverse_index(block_indices, block_counts, nblk, chunk_cap, window=window)
    obuf = torch.empty((B, N, HQ, S, D), dtype=obuf_dtype, device=q.device)
    lsebuf = torch.empty((B, N, HQ, S), dtype=torch.float32, device=q.device)
    bsa.bsa_fwd_kvouter(q, k, v, B, N, HQ, H, D, plan.row_ptr, plan.q_idx, plan.slot, plan.chunks,
                        plan.n_chunks, plan.max_chunks, nblk, block_size, S, causal, scale, obuf, lsebuf,
                        window=plan.window)
    out = torch.empty_like(q)
    lse = torch.empty((B, N, HQ), dtype=torch.float32, device=q.device) if need_lse else None
    bsa.bsa_combine(obuf, lsebuf, block_counts, B, N, HQ, H, S, D, out, lse)
    return out, lse, plan, obuf, lsebuf


def effective_flops(hq, n, d, k, bk, batch=1):
    """The metric's FLOP count 4*Hq*N*d*k*B_k ("MSA ... KV-outer" page, eq. 13/15)."""
    return 4.0 * batch * hq * n * d * k * bk


def ceil_div(a, b):
    return -(-a // b)


# ---------------------------------------------------------------- token serving over the paged 4-bit cache

class CacheStep(NamedTuple):
    """What one serving step's tables hold: the pool's new count, each request's
    first new token [R + 1], and each new token's request, position and slot
    [max_tokens] (-1 behind the last)."""
    pool_count: torch.Tensor
    query_start: torch.Tensor
    token_req: torch.Tensor
    token_pos: torch.Tensor
    slots: torch.Tensor


def new_cache(n_pages, H, page_size, D, device="cuda"):
    """An empty paged 4-bit cache, uint8 [n_pages, H, page_size / 16, 18 D]."""
    if not bsa.bsa_cache_bytes(n_pages, H, page_size, D):
        raise ValueError("no cache of %d pages of %d tokens, %d heads of %d channels" % (n_pages, page_size, H, D))
    return torch.zeros((n_pages, H, page_size // 16, 18 * D), dtype=torch.uint8, device=device)


def cache_tables(old_lens, new_lens, page_size, block_table, pool, pool_count, max_tokens, out=None):
    """Block tables [R, max_pages] and page pool from old_lens to new_lens (both int32 [R]), in place, and the
    step's new tokens.  A step that cannot be served sets new_lens back to old_lens.  ``out``: the five tensors of
    the result, to be written instead of new ones (its first may be pool_count)."""
    R, max_pages = block_table.shape
    dev = block_table.device
    if out is None:
        tok = torch.empty(2, max_tokens, dtype=torch.int32, device=dev)
        out = (torch.empty(1, dtype=torch.int32, device=dev),
               torch.empty(R + 1, dtype=torch.int32, device=dev), tok[0], tok[1],
               torch.empty(max_tokens, dtype=torch.int64, device=dev))
    nbytes = bsa.bsa_cache_tables_workspace(R)
    ws = torch.empty(nbytes // 4, dtype=torch.int32, device=dev) if nbytes else None
    bsa.bsa_cache_tables(old_lens, new_lens, R, page_size, block_table, max_pages, pool, pool.shape[0], pool_count,
                         *out, max_tokens, ws)
    return CacheStep(*out)


def _check_rows(name, t, T, *rest):
    """A tensor [T or more, *rest]: others may have as many elements, and would be read as other rows."""
    if t is not None and (t.shape[1:] != rest or t.shape[0] < T):
        raise ValueError("%s: a tensor %s is needed, got %s" % (name, [T, *rest], tuple(t.shape)))


def _check_scales(k_scale, v_scale, H):
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if t is not None and t.numel() != H:
            raise ValueError("%s: a scale for each of %d KV heads is needed, got %s" % (name, H, tuple(t.shape)))


def cache_append(k, v, slots, cache, k_scale=None, v_scale=None, values=None):
    """K and V rows [T, H, D] (token stride free) rounded to 4 bits into their slots of the cache.  ``values``: a
    pair of [T, H, D] tensors (or longer ones) that receive the rows as the cache holds them."""
    T, H, D = k.shape
    if cache.shape[1] != H or cache.shape[3] != 18 * D:
        raise ValueError("cache %s does not hold %d heads of %d channels" % (tuple(cache.shape), H, D))
    if (k_scale is not None and k_scale.numel() != H) or (v_scale is not None and v_scale.numel() != H):
        _check_scales(k_scale, v_scale, H)
    kv, vv = (None, None) if values is None else values
    if values is not None and (kv is None or vv is None or kv.shape != k.shape or vv.shape != k.shape):
        _check_rows("values", kv, T, H, D)
        _check_rows("values", vv, T, H, D)
    bsa.bsa_cache_append(k, v, T, H, D, slots, cache, cache.shape[0], cache.shape[2] * 16, k_scale, v_scale, kv, vv)


def cache_attention(q, cache, block_table, token_req, token_pos, k_scale=None, v_scale=None, block_indices=None,
                    block_counts=None, block_size=0, scale=None, need_lse=True):
    """Query rows [T, HQ, D] of the given requests and positions over the cached keys up to each row's own position:
    all of them, or with block_indices [T, H, S] / block_counts [T, H] those of the listed blocks.  Returns
    (out [T, HQ, D], lse [T, HQ] or None); rows of tokens with request -1 are not written."""
    T, HQ, D = q.shape
    n_pages, H, strips, width = cache.shape
    if width != 18 * D:
        raise ValueError("cache %s does not hold %d channels" % (tuple(cache.shape), D))
    R, max_pages = block_table.shape
    if (k_scale is not None and k_scale.numel() != H) or (v_scale is not None and v_scale.numel() != H):
        _check_scales(k_scale, v_scale, H)
    S = 0
    if block_indices is not None:
        S = block_indices.shape[-1]
        if block_indices.shape != (T, H, S) or block_counts is None or block_counts.shape != (T, H):
            _check_rows("block_indices", block_indices, T, H, S)
            _check_rows("block_counts", block_counts, T, H)
    max_keys = S * block_size if S else max_pages * strips * 16
    # (sizes one by one: as a tuple they take torch 1.6 us longer to parse, of the call's 20)
    out = torch.empty(T, HQ, D, dtype=q.dtype, device=q.device)
    lse = torch.empty(T, HQ, dtype=torch.float32, device=q.device) if need_lse else None
    nbytes = bsa.bsa_cache_attention_workspace(T, HQ, H, D, max_keys)
    ws = torch.empty(nbytes // 4, dtype=torch.float32, device=q.device) if nbytes else None
    bsa.bsa_fwd_cache_tokens(q, T, HQ, H, D, cache, n_pages, strips * 16, block_table, R, max_pages, token_req,
                             token_pos, k_scale, v_scale, block_indices, block_counts, S, block_size,
                             D ** -0.5 if scale is None else scale, out, lse, ws)
    return out, lse


class Rotary(NamedTuple):
    """Frequencies of a rotation: turns int64 [P] in 2^-64 turns a position, the axis
    of each (int32 [P], None with one axis) and the factor of cos and sin."""
    turns: torch.Tensor
    axis: Optional[torch.Tensor]
    factor: float

    def table(self, positions, out=None):
        return rotary_table(positions, self.turns, self.axis, self.factor, out)


def rotary_frequencies(channels, base=10000.0, sections=None, scaling=None, stretch=1.0, trained=0, ramp=(1.0, 32.0),
                       device="cuda"):
    """Frequencies of ``channels`` rotated channels: base^(-i / P) for pair i of P.  ``sections``: channels of each
    axis (they sum to ``channels``), every axis with a ladder of its own.  For contexts ``stretch`` times the
    ``trained`` positions, ``scaling`` is
      "linear"  every frequency / stretch
      "base"    base * stretch^(d / (d - 2)) over the axis's d channels: the highest frequency stays, the lowest is
                divided by stretch
      "parts"   frequencies of fewer than ramp[0] turns in ``trained`` positions / stretch, those of more than ramp[1]
                as they are, linear between the two; cos and sin times 0.1 ln(stretch) + 1."""
    if scaling not in (None, "linear", "base", "parts"):
        raise ValueError("no scaling %r" % (scaling,))
    sections = [channels] if sections is None else list(sections)
    if sum(sections) != channels or any(d < 2 or d % 2 for d in sections):
        raise ValueError("sections %s: even numbers that sum to %d are needed" % (sections, channels))
    if not stretch >= 1.0 or (scaling == "parts" and not (trained > 0 and ramp[1] > ramp[0])):
        raise ValueError("stretch must be at least 1, and scaling by parts needs trained positions and a rising ramp")
    turns, axis = [], []
    for a, d in enumerate(sections):
        own = base * stretch ** (d / (d - 2)) if scaling == "base" and d > 2 else base
        for i in range(d // 2):
            f = own ** (-2 * i / d) / (2 * math.pi)  # turns a position
            if scaling == "linear":
                f /= stretch
            elif scaling == "parts":
                kept = min(1.0, max(0.0, (f * trained - ramp[0]) / (ramp[1] - ramp[0])))
                f = f * kept + f / stretch * (1.0 - kept)
            t = round(f * 2.0 ** 64) % (1 << 64)
            turns.append(t - (1 << 64) if t >> 63 else t)
            axis.append(a)
    return Rotary(torch.tensor(turns, dtype=torch.int64, device=device),
                  torch.tensor(axis, dtype=torch.int32, device=device) if len(sections) > 1 else None,
                  0.1 * math.log(stretch) + 1.0 if scaling == "parts" else 1.0)


def rotary_table(positions, turns, axis=None, factor=1.0, out=None):
    """(cos, sin) float32 [T, P] of positions int32 [T] or [T, axes] and the frequencies of ``Rotary``."""
    shape = positions.shape
    if not 1 <= len(shape) <= 2 or turns.dim() != 1:
        raise ValueError("positions [T] or [T, axes] and turns [P] are needed, got %s and %s" % (tuple(shape), tuple(turns.shape)))
    T, axes = shape if len(shape) == 2 else (shape[0], 1)
    P = turns.shape[0]
    if axis is not None and axis.shape != turns.shape:
        raise ValueError("axis: one for each of %d frequencies is needed, got %s" % (P, tuple(axis.shape)))
    if out is None:
        dev = turns.device
        out = (torch.empty(T, P, dtype=torch.float32, device=dev), torch.empty(T, P, dtype=torch.float32, device=dev))
    elif out[0].shape != (T, P) or out[1].shape != (T, P):
        raise ValueError("out: two tensors [%d, %d] are needed" % (T, P))
    bsa.bsa_rotary_table(positions, T, axes, turns, axis, P, factor, out[0], out[1])
    return out


def rotate(q, k, cos, sin, interleaved=False, q_weight=None, k_weight=None, eps=1e-6, heads_first=False,
           transpose=False, out=None):
    """q [B, T, HQ, D] and k [B, T, H, D] (or both without B; k may be None) rotated by cos and sin [T, P] ([B, T, P]:
    of each sequence), after an RMS norm over each head's channels where there is a weight [D].  Any strides with
    adjacent channels.  Returns (q, k) as new tensors of the same layout, or heads first ([B, H, T, D], what the
    block-sparse stages read).  ``transpose``: the transposed rotation, which is the gradient's and takes a rotation
    back.  ``out``: the two tensors to write instead of new ones, q and k themselves among them (with their own strides)."""
    shape, flat = q.shape, q.dim() == 3
    B, T, HQ, D = (1, *shape) if flat else shape
    H, P = 0 if k is None else k.shape[-2], cos.shape[-1]
    if sin.shape != cos.shape or (cos.shape != (T, P) and cos.shape != (B, T, P)):
        raise ValueError("tables [%d, P] or [%d, %d, P] are needed, got %s and %s"
                         % (T, B, T, tuple(cos.shape), tuple(sin.shape)))
    if (q_weight is not None and q_weight.shape != (D,)) or (k_weight is not None and k_weight.shape != (D,)):
        raise ValueError("q_weight, k_weight: [%d] is needed" % D)
    if out is None:
        dt, dev = q.dtype, q.device
        if heads_first:
            out = (torch.empty(*shape[:-3], HQ, T, D, dtype=dt, device=dev),
                   None if k is None else torch.empty(*shape[:-3], H, T, D, dtype=dt, device=dev))
        else:
            out = (torch.empty(*shape, dtype=dt, device=dev),
                   None if k is None else torch.empty(*shape[:-2], H, D, dtype=dt, device=dev))
    bsa.bsa_rotate(q, k, B, T, HQ, H, D, P, cos, sin, T * P if cos.dim() == 3 else 0, out[0], out[1], interleaved,
                   transpose, q_weight, k_weight, eps, heads_first)
    return out


def cache_append_rotated(k, v, slots, cache, cos, sin, k_scale=None, v_scale=None, interleaved=False, values=None,
                         q=None, q_out=None):
    """``cache_append`` with K rotated on the way by cos and sin [T, P], and the queries q [T, HQ, D] rotated in the
    same launch into ``q_out`` (a new tensor if None), which is returned."""
    T, H, D = k.shape
    if cache.shape[1] != H or cache.shape[3] != 18 * D:
        raise ValueError("cache %s does not hold %d heads of %d channels" % (tuple(cache.shape), H, D))
    P = cos.shape[-1]
    if cos.shape != (T, P) or sin.shape != (T, P):
        raise ValueError("tables [%d, P] are needed, got %s and %s" % (T, tuple(cos.shape), tuple(sin.shape)))
    if (k_scale is not None and k_scale.numel() != H) or (v_scale is not None and v_scale.numel() != H):
        _check_scales(k_scale, v_scale, H)
    kv, vv = (None, None) if values is None else values
    if values is not None and (kv is None or vv is None or kv.shape != k.shape or vv.shape != k.shape):
        _check_rows("values", kv, T, H, D)
        _check_rows("values", vv, T, H, D)
    HQ = 0
    if q is not None:
        HQ = q.shape[1]
        if q_out is None:
            q_out = torch.empty(T, HQ, D, dtype=q.dtype, device=q.device)
        elif q_out.shape != q.shape:
            _check_rows("q_out", q_out, T, HQ, D)
    elif q_out is not None:
        raise ValueError("q_out without q")
    bsa.bsa_cache_append_rotated(k, v, T, H, D, slots, cache, cache.shape[0], cache.shape[2] * 16, k_scale, v_scale, kv,
                                 vv, cos, sin, P, interleaved, q, HQ, q_out)
    return q_out


def cross_attention(q, k, v, key_lens=None, query_start=None, key_start=None, scale=None, need_lse=True, out=None,
                    lse=None):
    """Queries over an encoder's states.  Padded: q [B, N, HQ, D], k and v [B, M, H, D], the first key_lens[b]
    (int32 [B], None: all) states of sequence b count.  Packed: q [N, HQ, D] with query_start, k and v [M, H, D] with
    key_start (int32 [B + 1] each; either alone or both).  Any strides with adjacent channels.  Returns
    (out as q, lse [B, N, HQ] or [N, HQ], or None).  ``out``, ``lse``: tensors to write instead of new ones; rows of
    no sequence are left as they were."""
    packed_q, packed_k, qshape, kshape = query_start is not None, key_start is not None, q.shape, k.shape
    if len(qshape) != (3 if packed_q else 4) or len(kshape) != (3 if packed_k else 4) or v.shape != kshape:
        raise ValueError("q %s, k %s, v %s: packed rows have three dimensions, padded ones four"
                         % (tuple(qshape), tuple(kshape), tuple(v.shape)))
    if packed_q:
        if query_start.dim() != 1:
            raise ValueError("query_start: [B + 1] is needed, got %s" % (tuple(query_start.shape),))
        B = query_start.shape[0] - 1
        N, HQ, D = qshape
    else:
        B, N, HQ, D = qshape
    M, H = kshape[-3], kshape[-2]
    if packed_k and key_start.dim() != 1:
        raise ValueError("key_start: [B + 1] is needed, got %s" % (tuple(key_start.shape),))
    if (packed_k and key_start.shape[0] - 1 != B) or (key_lens is not None and key_lens.shape != (B,)):
        raise ValueError("the states of %d sequences are needed" % B)
    if out is None:
        out = torch.empty_like(q)
    if need_lse and lse is None:
        if packed_q:
            lse = torch.empty(N, HQ, dtype=torch.float32, device=q.device)
        elif q.stride(2) > q.stride(1):  # heads first, as q
            lse = torch.empty(B, HQ, N, dtype=torch.float32, device=q.device).transpose(1, 2)
        else:
            lse = torch.empty(B, N, HQ, dtype=torch.float32, device=q.device)
    nbytes = bsa.bsa_cross_workspace(q.dtype, B, N, M, HQ, H, D, packed_q, packed_k)
    ws = torch.empty(nbytes // 4, dtype=torch.float32, device=q.device) if nbytes else None
    bsa.bsa_fwd_cross(q, k, v, B, N, M, HQ, H, D, query_start, key_start, key_lens,
                      D ** -0.5 if scale is None else scale, out, lse, ws)
    return out, lse


class TokenCache:
    """One layer's paged 4-bit cache with its tables, for R requests.

    A serving step is ``step`` (the tables, from the requests' new lengths),
    ``append`` (the new tokens' K and V) and ``attend`` (their queries).  Several
    layers can share the tables: give the first layer's cache as ``tables``."""

    def __init__(self, R, n_pages, max_pages, H, D, page_size=64, k_scale=None, v_scale=None, device="cuda",
                 tables=None):
        self.page_size = page_size
        self.cache = new_cache(n_pages, H, page_size, D, device)
        self.k_scale, self.v_scale = k_scale, v_scale
        self._own = tables is None
        if self._own:
            self.lens = torch.zeros((R,), dtype=torch.int32, device=device)
            self.block_table = torch.full((R, max_pages), -1, dtype=torch.int32, device=device)
            self.pool = torch.arange(n_pages - 1, -1, -1, dtype=torch.int32, device=device)  # page 0 on top
            self.pool_count = torch.full((1,), n_pages, dtype=torch.int32, device=device)
        else:
            if tables.block_table.shape != (R, max_pages) or tables.page_size != page_size \
                    or tables.pool.shape[0] != n_pages:
                raise ValueError("the shared tables have other sizes")
            self.lens, self.block_table = tables.lens, tables.block_table
            self.pool, self.pool_count = tables.pool, tables.pool_count

    def step(self, new_lens, max_tokens):
        """The tables for new_lens int32 [R]; returns the CacheStep.  A step that cannot be served (too few
        free pages, more than max_tokens new tokens: BSA_ERR_CAPACITY on the device status) has no tokens and
        leaves tables and lengths as they were."""
        if not self._own:
            raise ValueError("these tables belong to another cache")
        if new_lens.shape != self.lens.shape:
            raise ValueError("the lengths of %d requests are needed, got %s" % (self.lens.shape[0], tuple(new_lens.shape)))
        held = new_lens.clone()
        R, dev = held.shape[0], held.device
        tok = torch.empty(2, max_tokens, dtype=torch.int32, device=dev)
        out = cache_tables(self.lens, held, self.page_size, self.block_table, self.pool, self.pool_count, max_tokens,
                           out=(self.pool_count, torch.empty(R + 1, dtype=torch.int32, device=dev), tok[0], tok[1],
                                torch.empty(max_tokens, dtype=torch.int64, device=dev)))
        self.lens.copy_(held)
        return out

    def append(self, k, v, step, values=None, rotary=None, interleaved=False, q=None):
        """The step's K and V into the cache.  ``rotary``: the step's (cos, sin) tables (``rotary_table`` of
        step.token_pos); K is then rotated on the way, and ``q`` [max_tokens, HQ, D], where given, is returned
        rotated."""
        if rotary is None:
            if q is not None:
                raise ValueError("queries are rotated by the rotary tables of the step")
            return cache_append(k, v, step.slots, self.cache, self.k_scale, self.v_scale, values)
        return cache_append_rotated(k, v, step.slots, self.cache, rotary[0], rotary[1], self.k_scale, self.v_scale,
                                    interleaved, values, q)

    def attend(self, q, step, block_indices=None, block_counts=None, block_size=0, scale=None, need_lse=True):
        return cache_attention(q, self.cache, self.block_table, step.token_req, step.token_pos, self.k_scale,
                               self.v_scale, block_indices, block_counts, block_size, scale, need_lse)
