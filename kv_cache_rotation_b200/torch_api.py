"""Marshalling helpers between torch tensors and the libkvq C ABI.

Nothing here computes: tensors are allocated with torch (device memory is
PyTorch's job), their addresses are put into the ABI structs, and the C entry
points run the CUDA kernels. Host-side tables (RoPE cos/sin, Lloyd-Max
levels) are filled by the library's own host helpers and uploaded.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import (KVQ_BF16, KVQ_F16, KVQ_FIELD_CODES, KVQ_FIELD_EXT, KVQ_FIELD_NORM, KVQ_FIELD_SCALE_ZERO, KVQ_FIELD_SINK,
               KVQ_Q_CODEBOOK, KVQ_Q_CODEBOOK_DYN, KVQ_Q_MINMAX, KVQ_ROT_FWHT_GROUP, KVQ_ROT_FWHT_HEAD, KVQ_ROT_ISO_SO3, KVQ_ROT_ISO_SO4, KVQ_ROT_NONE,
               check,
               kvq_decode, kvq_desc, kvq_encode, kvq_paged, kvq_lloyd_max_codebook, kvq_packed, kvq_packed_bytes,
               kvq_rope_table, kvq_score, kvq_score_literal, kvq_tables)

ROT = {"none": KVQ_ROT_NONE, "fwht_head": KVQ_ROT_FWHT_HEAD, "fwht_group": KVQ_ROT_FWHT_GROUP,
       "iso": KVQ_ROT_ISO_SO4, "iso3": KVQ_ROT_ISO_SO3}
QUANT = {"minmax": KVQ_Q_MINMAX, "codebook": KVQ_Q_CODEBOOK, "codebook_dyn": KVQ_Q_CODEBOOK_DYN}


def make_desc(*, batch, heads, head_dim=128, tokens, t0=0, t_cap=None, bits, group=128, group_heads=1, rope=0,
              n_sink=0, rot="fwht_head", quant="minmax") -> kvq_desc:
    d = kvq_desc()
    d.batch, d.heads, d.head_dim, d.tokens, d.t0 = batch, heads, head_dim, tokens, t0
    d.t_cap = t0 + tokens if t_cap is None else t_cap
    d.bits, d.group, d.group_heads, d.rope, d.n_sink = bits, group, group_heads, int(rope), n_sink
    d.rot = ROT[rot] if isinstance(rot, str) else rot
    d.quant = QUANT[quant] if isinstance(quant, str) else quant
    return d


@dataclass
class Packed:
    codes: torch.Tensor
    scale_zero: Optional[torch.Tensor]
    sink: Optional[torch.Tensor]
    norm: Optional[torch.Tensor]
    ext: Optional[torch.Tensor] = None

    def struct(self) -> kvq_packed:
        p = kvq_packed()
        p.codes = self.codes.data_ptr()
        p.scale_zero = self.scale_zero.data_ptr() if self.scale_zero is not None else None
        p.sink = self.sink.data_ptr() if self.sink is not None else None
        p.norm = self.norm.data_ptr() if self.norm is not None else None
        p.ext = self.ext.data_ptr() if self.ext is not None else None
        return p

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size()
                   for t in (self.codes, self.scale_zero, self.sink, self.norm, self.ext) if t is not None)


def alloc_packed(d: kvq_desc, device="cuda", zero=True) -> Packed:
    """Allocate the cache buffers of a descriptor (sizes from kvq_packed_bytes)."""
    alloc = torch.zeros if zero else torch.empty

    def buf(field, dtype, shape):
        n = kvq_packed_bytes(d, field)
        if n == 0:
            return None
        t = alloc(n, dtype=torch.uint8, device=device)
        return t.view(dtype).view(shape)

    B, H, C, D = d.batch, d.heads, d.t_cap, d.head_dim
    codes = buf(KVQ_FIELD_CODES, torch.uint8, (B, H, C, D * d.bits // 8))
    ng = D // d.group if d.quant == KVQ_Q_MINMAX else 0
    sz = buf(KVQ_FIELD_SCALE_ZERO, torch.int16, (B, H, C, ng, 2)) if ng else None
    sink = buf(KVQ_FIELD_SINK, torch.float16, (B, H, d.n_sink, D)) if d.n_sink else None
    norm = buf(KVQ_FIELD_NORM, torch.float32, (B, H, C))
    ext = buf(KVQ_FIELD_EXT, torch.int16, (B, H, C))
    return Packed(codes, sz, sink, norm, ext)


def rope_table(t_max: int, head_dim: int, device="cuda", base: float = 10000.0, freq: int = 0) -> torch.Tensor:
    """(cos, sin) table [t_max][head_dim/2][2] filled by kvq_rope_table_ex (freq: KVQ_ROPE_*)."""
    from . import kvq_rope_table_ex
    host = torch.empty((t_max, head_dim // 2, 2), dtype=torch.float32)
    check(kvq_rope_table_ex(host.data_ptr(), t_max, head_dim, base, freq), "kvq_rope_table_ex")
    return host.to(device)


def lloyd_max_codebook(bits: int, head_dim: int, device="cuda") -> torch.Tensor:
    host = torch.empty(1 << bits, dtype=torch.float32)
    check(kvq_lloyd_max_codebook(host.data_ptr(), bits, head_dim), "kvq_lloyd_max_codebook")
    return host.to(device)


@dataclass
class Tables:
    """Device tables of one call; holds the tensors so their memory stays
    alive for as long as the struct built from them is in use."""
    perm: Optional[torch.Tensor] = None
    rope_cs: Optional[torch.Tensor] = None
    qL: Optional[torch.Tensor] = None
    qR: Optional[torch.Tensor] = None
    codebook: Optional[torch.Tensor] = None
    sink_pos: Optional[torch.Tensor] = None  # int32 [B][n_sink]: the list form of the sink set
    codebook_wide: Optional[torch.Tensor] = None  # dynamic codebooks: the (bits+1)-bit N(0,1) levels
    ch_scale: Optional[torch.Tensor] = None  # dynamic codebooks: f32 [H][D]
    ch_wide: Optional[torch.Tensor] = None  # dynamic codebooks: int32 [H][D/32] outlier-channel masks

    def struct(self) -> kvq_tables:
        tb = kvq_tables()
        tb.perm = self.perm.data_ptr() if self.perm is not None else None
        tb.rope_cs = self.rope_cs.data_ptr() if self.rope_cs is not None else None
        tb.rope_rows = self.rope_cs.shape[0] if self.rope_cs is not None else 0
        tb.qL = self.qL.data_ptr() if self.qL is not None else None
        tb.qR = self.qR.data_ptr() if self.qR is not None else None
        tb.codebook = self.codebook.data_ptr() if self.codebook is not None else None
        if self.sink_pos is not None:
            _req(self.sink_pos, "sink_pos", (torch.int32,))
            tb.sink_pos = self.sink_pos.data_ptr()
        tb.codebook_wide = self.codebook_wide.data_ptr() if self.codebook_wide is not None else None
        tb.ch_scale = self.ch_scale.data_ptr() if self.ch_scale is not None else None
        tb.ch_wide = self.ch_wide.data_ptr() if self.ch_wide is not None else None
        return tb


def make_tables(perm=None, rope_cs=None, qL=None, qR=None, codebook=None, sink_pos=None, codebook_wide=None,
                ch_scale=None, ch_wide=None) -> Tables:
    return Tables(perm, rope_cs, qL, qR, codebook, sink_pos, codebook_wide, ch_scale, ch_wide)


def _req(t: torch.Tensor, name: str, dtypes, shape=None) -> None:
    """Reject a tensor the C ABI would misread: it must be a contiguous CUDA
    tensor of one of `dtypes`, shaped `shape` when given."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _kv_shape(d: kvq_desc):
    return (d.batch, d.heads, d.tokens, d.head_dim)


def _q_heads(d: kvq_desc, q: torch.Tensor) -> int:
    _req(q, "q", (torch.float16,))
    if q.dim() != 3 or q.shape[0] != d.batch or q.shape[2] != d.head_dim:
        raise ValueError(f"q: shape {tuple(q.shape)}, expected ({d.batch}, q_heads, {d.head_dim})")
    return int(q.shape[1])


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def encode(d: kvq_desc, x: torch.Tensor, tables: Tables, packed: Packed, stream=None) -> None:
    _req(x, "x", (torch.float16,), _kv_shape(d))
    check(kvq_encode(d, x.data_ptr(), tables.struct(), packed.struct(), _stream(stream)), "kvq_encode")


def decode(d: kvq_desc, packed: Packed, tables: Tables, out: torch.Tensor, stream=None) -> None:
    _req(out, "out", (torch.float16, torch.float32), _kv_shape(d))
    fp32 = 1 if out.dtype == torch.float32 else 0
    check(kvq_decode(d, packed.struct(), tables.struct(), out.data_ptr(), fp32, _stream(stream)), "kvq_decode")


def score(d: kvq_desc, q: torch.Tensor, packed: Packed, tables: Tables, n_tokens: int, scale: float,
          out: torch.Tensor, stream=None) -> None:
    hq = _q_heads(d, q)
    _req(out, "scores", (torch.float32,), (d.batch, hq, n_tokens))
    check(kvq_score(d, q.data_ptr(), hq, packed.struct(), tables.struct(), n_tokens, scale,
                    out.data_ptr(), _stream(stream)), "kvq_score")


def score_literal(d: kvq_desc, q: torch.Tensor, packed: Packed, tables: Tables, n_tokens: int, scale: float,
                  out: torch.Tensor, stream=None) -> None:
    """The scores of score(), every key decoded on the fly (the literal per-token form)."""
    hq = _q_heads(d, q)
    _req(out, "scores", (torch.float32,), (d.batch, hq, n_tokens))
    check(kvq_score_literal(d, q.data_ptr(), hq, packed.struct(), tables.struct(), n_tokens, scale,
                            out.data_ptr(), _stream(stream)), "kvq_score_literal")


def attend_workspace(dk: kvq_desc, dv: kvq_desc, q_heads: int, n_tokens: int, device="cuda") -> torch.Tensor:
    """A workspace tensor for kvq_attend (256-byte aligned, as torch allocates)."""
    from . import kvq_attend_workspace_bytes
    nb = kvq_attend_workspace_bytes(dk, dv, q_heads, n_tokens)
    if nb == 0:
        raise ValueError("kvq_attend: invalid or unsupported shapes")
    return torch.empty(nb, dtype=torch.uint8, device=device)


def attend(dk: kvq_desc, dv: kvq_desc, q: torch.Tensor, k_packed: Packed, tk: Tables, v_packed: Packed, tv: Tables,
           n_tokens: int, scale: float, out: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    from . import kvq_attend
    hq = _q_heads(dk, q)
    _req(out, "out", (torch.float32,), (dk.batch, hq, dk.head_dim))
    _req(workspace, "workspace", (torch.uint8,))
    check(kvq_attend(dk, dv, q.data_ptr(), hq, k_packed.struct(), tk.struct(), v_packed.struct(),
                     tv.struct(), n_tokens, scale, out.data_ptr(), workspace.data_ptr(), workspace.numel(),
                     _stream(stream)), "kvq_attend")


def attend_noalloc(dk: kvq_desc, dv: kvq_desc, q: torch.Tensor, k_packed: Packed, tk: Tables, v_packed: Packed,
                   tv: Tables, n_tokens: int, scale: float, out: torch.Tensor, stream=None) -> None:
    """kvq_attend through the library's fixed scratch (no workspace tensor)."""
    from . import kvq_attend_noalloc
    hq = _q_heads(dk, q)
    _req(out, "out", (torch.float32,), (dk.batch, hq, dk.head_dim))
    check(kvq_attend_noalloc(dk, dv, q.data_ptr(), hq, k_packed.struct(), tk.struct(), v_packed.struct(),
                             tv.struct(), n_tokens, scale, out.data_ptr(), _stream(stream)), "kvq_attend_noalloc")


def calibrate_workspace(d: kvq_desc, device="cuda") -> torch.Tensor:
    """A workspace tensor for kvq_calibrate_perm."""
    from . import kvq_calibrate_workspace_bytes
    nb = kvq_calibrate_workspace_bytes(d)
    if nb == 0:
        raise ValueError("kvq_calibrate_perm: invalid or unsupported descriptor")
    return torch.empty(nb, dtype=torch.uint8, device=device)


def calibrate_perm(d: kvq_desc, x: torch.Tensor, tb: Tables, perm_out: torch.Tensor = None,
                   workspace: torch.Tensor = None, stream=None) -> torch.Tensor:
    """Channel permutation by abs-max (int16 [H][head_dim]) for kvq_tables.perm."""
    from . import kvq_calibrate_perm
    _req(x, "x", (torch.float16,), _kv_shape(d))
    if perm_out is None:
        perm_out = torch.empty((d.heads, d.head_dim), dtype=torch.int16, device=x.device)
    if workspace is None:
        workspace = calibrate_workspace(d, x.device)
    _req(perm_out, "perm_out", (torch.int16,), (d.heads, d.head_dim))
    check(kvq_calibrate_perm(d, x.data_ptr(), tb.struct(), perm_out.data_ptr(), workspace.data_ptr(),
                             workspace.numel(), _stream(stream)), "kvq_calibrate_perm")
    return perm_out


def calibrate_codebook(d: kvq_desc, x: torch.Tensor, tb: Tables, ch_scale: torch.Tensor = None,
                       ch_wide: torch.Tensor = None, workspace: torch.Tensor = None, stream=None):
    """Dynamic codebook tables (ch_scale f32 [H][D], ch_wide int32 [H][D/32] bit masks) for
    Tables.ch_scale / Tables.ch_wide."""
    from . import kvq_calibrate_codebook, kvq_calibrate_codebook_workspace_bytes
    _req(x, "x", (torch.float16,), _kv_shape(d))
    if ch_scale is None:
        ch_scale = torch.empty((d.heads, d.head_dim), dtype=torch.float32, device=x.device)
    if ch_wide is None:
        ch_wide = torch.empty((d.heads, d.head_dim // 32), dtype=torch.int32, device=x.device)
    if workspace is None:
        nb = kvq_calibrate_codebook_workspace_bytes(d)
        if nb == 0:
            raise ValueError("kvq_calibrate_codebook: invalid or unsupported descriptor")
        workspace = torch.empty(nb, dtype=torch.uint8, device=x.device)
    _req(ch_scale, "ch_scale", (torch.float32,), (d.heads, d.head_dim))
    _req(ch_wide, "ch_wide", (torch.int32,), (d.heads, d.head_dim // 32))
    check(kvq_calibrate_codebook(d, x.data_ptr(), tb.struct(), ch_scale.data_ptr(), ch_wide.data_ptr(),
                                 workspace.data_ptr(), workspace.numel(), _stream(stream)), "kvq_calibrate_codebook")
    return ch_scale, ch_wide


def detect_sinks_workspace(d: kvq_desc, device="cuda") -> torch.Tensor:
    """A workspace tensor for kvq_detect_sinks."""
    from . import kvq_detect_sinks_workspace_bytes
    nb = kvq_detect_sinks_workspace_bytes(d)
    if nb == 0:
        raise ValueError("kvq_detect_sinks: invalid descriptor")
    return torch.empty(nb, dtype=torch.uint8, device=device)


def detect_sinks(d: kvq_desc, x: torch.Tensor, *, tau: float, max_sinks: int, sink_pos: torch.Tensor = None,
                 count: torch.Tensor = None, workspace: torch.Tensor = None, stream=None):
    """Attention sinks by massive activations: (sink_pos int32 [B][max_sinks], ascending
    positions padded with -1, for Tables.sink_pos with n_sink = max_sinks; count int32 [B])."""
    from . import kvq_detect_sinks
    _req(x, "x", (torch.float16,), _kv_shape(d))
    if sink_pos is None:
        sink_pos = torch.empty((d.batch, max_sinks), dtype=torch.int32, device=x.device)
    if count is None:
        count = torch.empty((d.batch,), dtype=torch.int32, device=x.device)
    if workspace is None:
        workspace = detect_sinks_workspace(d, x.device)
    _req(sink_pos, "sink_pos", (torch.int32,), (d.batch, max_sinks))
    _req(count, "count", (torch.int32,), (d.batch,))
    check(kvq_detect_sinks(d, x.data_ptr(), float(tau), int(max_sinks), sink_pos.data_ptr(), count.data_ptr(),
                           workspace.data_ptr(), workspace.numel(), _stream(stream)), "kvq_detect_sinks")
    return sink_pos, count


def bind_detect_sinks(d: kvq_desc, x: torch.Tensor, tau: float, sink_pos: torch.Tensor, count: torch.Tensor,
                      workspace: torch.Tensor, stream=None):
    from . import lib
    _req(x, "x", (torch.float16,), _kv_shape(d))
    _req(sink_pos, "sink_pos", (torch.int32,))
    _req(count, "count", (torch.int32,), (d.batch,))
    if sink_pos.dim() != 2 or sink_pos.shape[0] != d.batch:
        raise ValueError(f"sink_pos: shape {tuple(sink_pos.shape)}, expected ({d.batch}, max_sinks)")
    st = _stream(stream)
    args = (ctypes.byref(d), x.data_ptr(), float(tau), int(sink_pos.shape[1]), sink_pos.data_ptr(),
            count.data_ptr(), workspace.data_ptr(), workspace.numel(), st)
    keep = (d, x, sink_pos, count, workspace)

    def call():
        check(lib.kvq_detect_sinks(*args), "kvq_detect_sinks")
    call.keep = keep
    return call


def pair_energy(d: kvq_desc, x: torch.Tensor, stream=None):
    """Exact RoPE-pair energies (uint64 [H][head_dim/2][2]: low, high words of the count of
    2^-48) and the pairs ranked by descending energy (int16 [H][head_dim/2])."""
    from . import kvq_pair_energy
    _req(x, "x", (torch.float16,), _kv_shape(d))
    energy = torch.empty((d.heads, d.head_dim // 2, 2), dtype=torch.uint64, device=x.device)
    rank = torch.empty((d.heads, d.head_dim // 2), dtype=torch.int16, device=x.device)
    check(kvq_pair_energy(d, x.data_ptr(), energy.data_ptr(), rank.data_ptr(), _stream(stream)), "kvq_pair_energy")
    return energy, rank


def bind_pair_energy(d: kvq_desc, x: torch.Tensor, energy: torch.Tensor, rank: torch.Tensor, stream=None):
    from . import lib
    _req(x, "x", (torch.float16,), _kv_shape(d))
    _req(energy, "energy", (torch.uint64,), (d.heads, d.head_dim // 2, 2))
    _req(rank, "rank", (torch.int16,), (d.heads, d.head_dim // 2))
    st = _stream(stream)
    args = (ctypes.byref(d), x.data_ptr(), energy.data_ptr(), rank.data_ptr(), st)
    keep = (d, x, energy, rank)

    def call():
        check(lib.kvq_pair_energy(*args), "kvq_pair_energy")
    call.keep = keep
    return call


def bind_calibrate(d: kvq_desc, x: torch.Tensor, tb: Tables, perm_out: torch.Tensor, workspace: torch.Tensor,
                   stream=None):
    from . import lib
    _req(x, "x", (torch.float16,), _kv_shape(d))
    _req(perm_out, "perm_out", (torch.int16,), (d.heads, d.head_dim))
    tbs, st = tb.struct(), _stream(stream)
    args = (ctypes.byref(d), x.data_ptr(), ctypes.byref(tbs), perm_out.data_ptr(), workspace.data_ptr(),
            workspace.numel(), st)
    keep = (d, x, tb, tbs, perm_out, workspace)

    def call():
        check(lib.kvq_calibrate_perm(*args), "kvq_calibrate_perm")
    call.keep = keep
    return call


def bind_attend(dk: kvq_desc, dv: kvq_desc, q: torch.Tensor, k_packed: Packed, tk: Tables, v_packed: Packed,
                tv: Tables, n_tokens: int, scale: float, out: torch.Tensor, workspace: torch.Tensor, stream=None):
    from . import lib
    hq = _q_heads(dk, q)
    _req(out, "out", (torch.float32,), (dk.batch, hq, dk.head_dim))
    _req(workspace, "workspace", (torch.uint8,))
    tks, kps, tvs, vps, st = tk.struct(), k_packed.struct(), tv.struct(), v_packed.struct(), _stream(stream)
    args = (ctypes.byref(dk), ctypes.byref(dv), q.data_ptr(), hq, ctypes.byref(kps), ctypes.byref(tks),
            ctypes.byref(vps), ctypes.byref(tvs), n_tokens, ctypes.c_float(scale), out.data_ptr(),
            workspace.data_ptr(), workspace.numel(), st)
    keep = (dk, dv, q, k_packed, tk, v_packed, tv, out, workspace, tks, kps, tvs, vps)

    def call():
        check(lib.kvq_attend(*args), "kvq_attend")
    call.keep = keep
    return call


# ---------------------------------------------------------------- the paged cache
@dataclass
class Paged:
    """A ragged batch over a paged cache (kvq_paged): int32 device tensors, filled by page_map or by
    the caller. What a call does not read may be None (the row maps for attend_paged, the lengths
    and the table for encode_paged and decode_paged)."""
    cu_rows: Optional[torch.Tensor] = None      # [S+1]
    kv_len: Optional[torch.Tensor] = None       # [S]
    block_table: Optional[torch.Tensor] = None  # [S][max_pages]
    seq: Optional[torch.Tensor] = None          # [n_rows]
    pos: Optional[torch.Tensor] = None          # [n_rows]
    slot: Optional[torch.Tensor] = None         # [n_rows]
    sink_slot: Optional[torch.Tensor] = None    # [S]: rows of the sink buffers (None: row s)

    def struct(self, n_rows: int = None, sink: Optional[torch.Tensor] = None) -> kvq_paged:
        S = None
        for t, name in ((self.kv_len, "kv_len"), (self.cu_rows, "cu_rows"), (self.block_table, "block_table"),
                        (self.sink_slot, "sink_slot")):
            if t is not None:
                n = t.shape[0] - (1 if name == "cu_rows" else 0)
                _req(t, name, (torch.int32,))
                if t.dim() != (2 if name == "block_table" else 1) or n < 0 or S not in (None, n):
                    raise ValueError(f"{name}: shape {tuple(t.shape)} does not fit {S} sequences")
                S = n
        for t, name in ((self.seq, "seq"), (self.pos, "pos"), (self.slot, "slot")):
            if t is not None:
                if n_rows is None:
                    n_rows = t.numel()
                _req(t, name, (torch.int32,), (n_rows,))
        p = kvq_paged()
        p.n_seqs, p.n_rows = S or 0, n_rows or 0
        p.max_pages = self.block_table.shape[1] if self.block_table is not None else 1
        p.sink_rows = sink.shape[0] if sink is not None else 0
        for name in ("cu_rows", "kv_len", "block_table", "seq", "pos", "slot", "sink_slot"):
            t = getattr(self, name)
            setattr(p, name, t.data_ptr() if t is not None else None)
        return p


def make_paged(n_seqs: int, n_rows: int, max_pages: int, block_table: torch.Tensor = None, sink_slot=None,
               device="cuda") -> Paged:
    """The arrays of a batch for page_map to fill (an empty block table is one of -1)."""
    def ints(*shape):
        return torch.empty(shape, dtype=torch.int32, device=device)
    if block_table is None:
        block_table = torch.full((n_seqs, max_pages), -1, dtype=torch.int32, device=device)
    return Paged(ints(n_seqs + 1), ints(n_seqs), block_table, ints(n_rows), ints(n_rows), ints(n_rows), sink_slot)


def alloc_paged(d: kvq_desc, sink_rows: int = 0, device="cuda", zero=True) -> Packed:
    """The buffers of a paged cache: d.batch pages of d.t_cap tokens, and the fp16 sinks of
    sink_rows sequences."""
    bare = kvq_desc.from_buffer_copy(d)
    bare.n_sink = 0
    p = alloc_packed(bare, device, zero)
    if d.n_sink:
        p.sink = (torch.zeros if zero else torch.empty)((sink_rows, d.heads, d.n_sink, d.head_dim), dtype=torch.float16,
                                                        device=device)
    return p


def _tensors(*things) -> list:
    """The tensors of a call's arguments: of tensors, batches, caches and tables."""
    out = []
    for x in things:
        if isinstance(x, torch.Tensor):
            out.append(x)
        elif isinstance(x, (Paged, Packed, Tables)):
            out += [t for t in vars(x).values() if t is not None]
    return out


def _here(tensors) -> None:
    """The library launches on the current device: all that a call reads or writes has to be there."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{dev}")


def _pool(d: kvq_desc, packed: Packed) -> None:
    """The buffers of a paged cache have the descriptor's sizes: the kernels count on them."""
    H, D, n_sink = d.heads, d.head_dim, d.n_sink
    records = d.batch * H * d.t_cap
    for t, name, each in ((packed.codes, "codes", D * d.bits // 8), (packed.scale_zero, "scale_zero", D // max(d.group, 1) * 4)):
        if t is not None:
            _req(t, name, (t.dtype,))
            if t.nbytes < records * each:
                raise ValueError(f"{name}: {t.nbytes} bytes, the descriptor needs {records * each}")
    if n_sink > 0 and packed.sink is not None:
        _req(packed.sink, "sink", (torch.float16,))
        if tuple(packed.sink.shape[1:]) != (H, n_sink, D):
            raise ValueError(f"sink: shape {tuple(packed.sink.shape)}, expected (sink_rows, {H}, {n_sink}, {D})")


def _row_tables(d: kvq_desc, tables: Tables) -> None:
    """The tables that the rows of a head-variant cache read."""
    if tables.perm is not None:
        _req(tables.perm, "perm", (torch.int16,))
        if tables.perm.numel() != d.heads * d.head_dim:
            raise ValueError(f"perm: shape {tuple(tables.perm.shape)}, expected ({d.heads}, {d.head_dim})")
    if d.rope and tables.rope_cs is not None:
        _req(tables.rope_cs, "rope_cs", (torch.float32,))
        if tables.rope_cs.numel() != tables.rope_cs.shape[0] * d.head_dim:
            raise ValueError(f"rope_cs: shape {tuple(tables.rope_cs.shape)}, expected (rows, {d.head_dim // 2}, 2)")


def _span(t: torch.Tensor):
    """First byte of a tensor, and the byte behind its last."""
    a, n = t.data_ptr(), t.numel()
    if n and not t.is_contiguous():
        n = 1 + sum((d - 1) * s for d, s in zip(t.shape, t.stride()))
    return a, a + n * t.element_size()


def _meet(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two tensors, dense ones or packed rows with a stride, share memory: slices of one projection do not,
    though they lie between each other (with different strides whatever lies so counts as shared)."""
    (a0, a1), (b0, b1) = _span(a), _span(b)
    if a0 == a1 or b0 == b1 or a0 >= b1 or b0 >= a1:
        return False
    fars = {t.stride(0) * t.element_size() for t in (a, b) if t.shape[0] > 1}
    if len(fars) != 1:
        return True
    far, off = fars.pop(), b0 - a0  # bytes between rows; where b's rows begin behind a's
    one, two = (t.nbytes // t.shape[0] for t in (a, b))
    return off % far < one or off % far + two > far


def _apart(writes: dict, reads) -> None:
    """No tensor that a call writes shares memory with one that it reads, or with another one that it writes."""
    outs = {n: t for n, t in writes.items() if t is not None}
    spans = sorted([(*_span(t), True) for t in outs.values()] + [(*_span(t), False) for t in reads])
    end = written = 0  # of all spans so far, and of the written ones
    for a, e, w in spans:
        if a < e and (a < written or (w and a < end)):
            break
        end, written = max(end, e), max(written, e) if w else written
    else:
        return  # nearly always; what follows is for spans that lie between each other
    names = list(outs)
    for i, name in enumerate(names):
        for u in (*reads, *(outs[o] for o in names[i + 1:])):
            if _meet(outs[name], u):
                raise ValueError(f"{name}: an output must not overlap what the call reads or writes beside it")


def _rows(t: torch.Tensor, name: str, dtypes, heads=None, dim=None) -> int:
    """Elements between the packed rows of t [n_rows][heads][dim]; the rows themselves are dense."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
    if t.dim() != 3 or (heads is not None and t.shape[1] != heads) or (dim is not None and t.shape[2] != dim):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected (n_rows, {heads or 'heads'}, {dim or 'head_dim'})")
    if (t.stride(2) != 1 and t.shape[2] > 1) or (t.stride(1) != t.shape[2] and t.shape[1] > 1):
        raise ValueError(f"{name}: the heads of a row must be dense")
    if t.shape[0] <= 1:  # a single row has any stride
        return -(-t.shape[1] * t.shape[2] // 8) * 8
    return int(t.stride(0))


def _new(shape, dtype, device, stream) -> torch.Tensor:
    """A tensor that a call on `stream` writes: its memory is that stream's, so that nothing which the current
    stream still has to do with a freed tensor's memory meets the call."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    own = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(_stream(stream), device=device)
    with torch.cuda.stream(own):
        return torch.empty(shape, dtype=dtype, device=device)


def _call(name: str, args: tuple, keep: tuple, stream, why=None):
    """A zero-argument call of the entry point `name`: on `stream`, or on the stream that is current
    when it is called (so a bound call can be captured). The arguments are converted here, once: the
    call costs the library's own time and about 2 us. It is refused on another current device."""
    from . import KVQ_OK, lib
    types = getattr(lib, name).argtypes
    fn = lib[name]  # a handle without argtypes: the converted arguments pass as they are
    fn.restype = ctypes.c_int32
    for t, a in zip(types, args):
        if t is ctypes.c_int32 and not -1 << 31 <= a < 1 << 31:  # ctypes would take the low bits
            raise ValueError(f"{name}: {a} does not fit 32 bits")
    args = tuple(t(a) if isinstance(a, (int, float)) else a for t, a in zip(types, args))
    fixed = None if stream is None else ctypes.c_void_p(_stream(stream))
    dev = torch.cuda.current_device()
    others = torch.cuda.device_count() > 1  # else no other device can be current, and asking costs 1 us

    def call():
        if others and torch.cuda.current_device() != dev:
            raise ValueError(f"{name}: bound on cuda:{dev}, called on cuda:{torch.cuda.current_device()}")
        status = fn(*args, fixed if fixed is not None else ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(dev)))
        if status != KVQ_OK:
            if why is not None:
                why()
            check(status, name)
    call.keep = (keep, _tensors(*keep))  # the tensors themselves: a field of a batch or cache may get another one
    return call


def bind_page_map(d: kvq_desc, batch: Paged, ctx_len: torch.Tensor, new_len: torch.Tensor, free_pages: torch.Tensor,
                  free_used: torch.Tensor, report: torch.Tensor, stream=None):
    d = kvq_desc.from_buffer_copy(d)  # here and below: the call is made with what was checked
    p = batch.struct()
    for name in ("cu_rows", "kv_len", "block_table", "seq", "pos", "slot"):
        if getattr(batch, name) is None:
            raise ValueError(f"{name}: page_map fills it")
    _req(ctx_len, "ctx_len", (torch.int32,), (p.n_seqs,))
    _req(new_len, "new_len", (torch.int32,), (p.n_seqs,))
    _req(free_pages, "free_pages", (torch.int32,), (free_pages.numel(),))
    _req(free_used, "free_used", (torch.int32,), (1,))
    _req(report, "report", (torch.int32,), (4,))
    _here(_tensors(batch, ctx_len, new_len, free_pages, free_used, report))
    args = (ctypes.byref(d), ctypes.byref(p), ctx_len.data_ptr(), new_len.data_ptr(), free_pages.data_ptr(),
            free_pages.numel(), free_used.data_ptr(), report.data_ptr())

    def why():  # the library refuses arrays that overlap, this says which
        reads = dict(ctx_len=ctx_len, new_len=new_len, free_pages=free_pages, free_used=free_used)
        writes = {n: getattr(batch, n) for n in ("cu_rows", "kv_len", "block_table", "seq", "pos", "slot")}
        writes["report"] = report
        for i, (name, t) in enumerate(writes.items()):
            for other, u in [*list(writes.items())[i + 1:], *reads.items()]:
                if _meet(t, u):
                    raise ValueError(f"{name}: written while {other} is read or written, they must not overlap")
    return _call("kvq_page_map", args, (d, p, batch, ctx_len, new_len, free_pages, free_used, report), stream, why)


def page_map(d: kvq_desc, batch: Paged, ctx_len: torch.Tensor, new_len: torch.Tensor, free_pages: torch.Tensor,
             free_used: torch.Tensor, report: torch.Tensor = None, stream=None) -> torch.Tensor:
    """Fill the batch from its lengths (kvq_page_map); returns the report, int32 [4]: rows, free pages
    taken in all, rows without a slot, pages that were lacking. report[1:2] is the next call's free_used, and
    batch.kv_len its ctx_len: copies of them where the next call writes the same tensors."""
    if report is None:
        report = _new((4,), torch.int32, ctx_len.device, stream)
    bind_page_map(d, batch, ctx_len, new_len, free_pages, free_used, report, stream)()
    return report


def bind_encode_paged(d: kvq_desc, x: torch.Tensor, batch: Paged, tables: Tables, packed: Packed, stream=None):
    d = kvq_desc.from_buffer_copy(d)
    stride = _rows(x, "x", (torch.float16,), d.heads, d.head_dim)
    p, tb, pk = batch.struct(x.shape[0], packed.sink), tables.struct(), packed.struct()
    _pool(d, packed), _row_tables(d, tables)
    reads = _tensors(x, batch, tables)
    _here(reads + _tensors(packed))
    _apart(dict(codes=packed.codes, scale_zero=packed.scale_zero, sink=packed.sink if d.n_sink else None), reads)
    args = (ctypes.byref(d), x.data_ptr(), stride, ctypes.byref(p), ctypes.byref(tb), ctypes.byref(pk))
    return _call("kvq_encode_paged", args, (d, x, batch, tables, packed, p, tb, pk), stream)


def encode_paged(d: kvq_desc, x: torch.Tensor, batch: Paged, tables: Tables, packed: Packed, stream=None) -> None:
    """Encode the rows x fp16 [n_rows][H][D] (dense heads, any row stride) into their slots, each slot one
    row's (the record of a slot given twice may be a mix of both rows')."""
    bind_encode_paged(d, x, batch, tables, packed, stream)()


def bind_decode_paged(d: kvq_desc, packed: Packed, batch: Paged, tables: Tables, out: torch.Tensor, stream=None):
    d = kvq_desc.from_buffer_copy(d)
    stride = _rows(out, "out", (torch.float16, torch.float32), d.heads, d.head_dim)
    p, tb, pk = batch.struct(out.shape[0], packed.sink), tables.struct(), packed.struct()
    _pool(d, packed), _row_tables(d, tables)
    reads = _tensors(batch, tables, packed)
    _here(reads + [out])
    _apart(dict(out=out), reads)
    args = (ctypes.byref(d), ctypes.byref(pk), ctypes.byref(p), ctypes.byref(tb), out.data_ptr(), stride,
            1 if out.dtype == torch.float32 else 0)
    return _call("kvq_decode_paged", args, (d, packed, batch, tables, out, p, tb, pk), stream)


def decode_paged(d: kvq_desc, packed: Packed, batch: Paged, tables: Tables, out: torch.Tensor, stream=None) -> None:
    """Decode the rows' records into out fp16 / fp32 [n_rows][H][D]; rows without a slot stay as they are."""
    bind_decode_paged(d, packed, batch, tables, out, stream)()


def attend_paged_workspace(dk: kvq_desc, dv: kvq_desc, q_heads: int, batch: Paged, max_rows: int, max_kv: int,
                           n_rows: int = None) -> torch.Tensor:
    """A workspace tensor for attend_paged; n_rows: the rows of q where the batch has no row maps."""
    from . import kvq_attend_paged_workspace_bytes
    p = batch.struct(n_rows)
    p.sink_rows = 1 << 30  # sizes alone count here
    nb = kvq_attend_paged_workspace_bytes(dk, dv, q_heads, p, max_rows, max_kv)
    if nb == 0:
        raise ValueError("kvq_attend_paged: invalid or unsupported shapes")
    return torch.empty(nb, dtype=torch.uint8, device=batch.cu_rows.device)


def bind_attend_paged(dk: kvq_desc, dv: kvq_desc, q: torch.Tensor, k_packed: Packed, tk: Tables, v_packed: Packed,
                      tv: Tables, batch: Paged, max_rows: int, max_kv: int, scale: float, out: torch.Tensor,
                      workspace: torch.Tensor, stream=None):
    dk, dv = kvq_desc.from_buffer_copy(dk), kvq_desc.from_buffer_copy(dv)
    qs = _rows(q, "q", (torch.float16,), None, dk.head_dim)
    os = _rows(out, "out", (torch.float16,), q.shape[1], dk.head_dim)
    if out.shape[0] != q.shape[0]:
        raise ValueError(f"out: {out.shape[0]} rows, expected {q.shape[0]}")
    _req(workspace, "workspace", (torch.uint8,))
    if (k_packed.sink is None) != (v_packed.sink is None) or \
            (k_packed.sink is not None and k_packed.sink.shape != v_packed.sink.shape):
        raise ValueError("sink: the two caches keep the sinks of the same sequences")
    p = batch.struct(q.shape[0], k_packed.sink)
    kp, vp, tks, tvs = k_packed.struct(), v_packed.struct(), tk.struct(), tv.struct()
    for d, pk, tb in ((dk, k_packed, tk), (dv, v_packed, tv)):
        _pool(d, pk), _row_tables(d, tb)
    reads = _tensors(q, batch, k_packed, tk, v_packed, tv)
    _here(reads + [out, workspace])
    _apart(dict(out=out, workspace=workspace), reads)
    args = (ctypes.byref(dk), ctypes.byref(dv), q.data_ptr(), qs, q.shape[1], ctypes.byref(kp), ctypes.byref(tks),
            ctypes.byref(vp), ctypes.byref(tvs), ctypes.byref(p), max_rows, max_kv, scale, out.data_ptr(), os,
            workspace.data_ptr(), workspace.numel())
    keep = (dk, dv, q, k_packed, tk, v_packed, tv, batch, out, workspace, p, kp, vp, tks, tvs)
    return _call("kvq_attend_paged", args, keep, stream)


def attend_paged(dk: kvq_desc, dv: kvq_desc, q: torch.Tensor, k_packed: Packed, tk: Tables, v_packed: Packed,
                 tv: Tables, batch: Paged, max_rows: int, max_kv: int, scale: float, out: torch.Tensor,
                 workspace: torch.Tensor, stream=None) -> None:
    """Causal attention of each sequence's new rows q fp16 [n_rows][q_heads][D] over its pages."""
    bind_attend_paged(dk, dv, q, k_packed, tk, v_packed, tv, batch, max_rows, max_kv, scale, out, workspace, stream)()


def bind_attend_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_rows: torch.Tensor, max_rows: int,
                       scale: float, out: torch.Tensor, stream=None):
    qs = _rows(q, "q", (torch.float16, torch.bfloat16))
    n, hq, dim = q.shape
    ks, vs = _rows(k, "k", (q.dtype,), None, dim), _rows(v, "v", (q.dtype,), k.shape[1], dim)
    os = _rows(out, "out", (q.dtype,), hq, dim)
    if not (k.shape[0] == v.shape[0] == out.shape[0] == n):
        raise ValueError("q, k, v and out must have the same rows")
    _req(cu_rows, "cu_rows", (torch.int32,))
    if cu_rows.dim() != 1 or cu_rows.numel() < 1:
        raise ValueError(f"cu_rows: shape {tuple(cu_rows.shape)}, expected (sequences + 1,)")
    _here((q, k, v, out, cu_rows))
    _apart(dict(out=out), (q, k, v, cu_rows))
    args = (q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, cu_rows.numel() - 1, n, hq, k.shape[1], dim,
            KVQ_BF16 if q.dtype == torch.bfloat16 else KVQ_F16, cu_rows.data_ptr(), max_rows, scale, out.data_ptr(), os)
    return _call("kvq_attend_prompt", args, (q, k, v, cu_rows, out), stream)


def attend_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_rows: torch.Tensor, max_rows: int,
                  scale: float, out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """Causal attention over packed prompts: q, out [n_rows][q_heads][D], k, v [n_rows][heads][D], all
    fp16 or all bf16, cu_rows int32 [S+1]. Rows that no sequence has, or beyond max_rows, are not written:
    where out is not given they hold whatever its memory held."""
    if out is None:
        out = _new(q.shape, q.dtype, q.device, stream)
    bind_attend_prompt(q, k, v, cu_rows, max_rows, scale, out, stream)()
    return out


# ---------------------------------------------------------------- pre-bound calls
# The same marshalling, done once: the returned zero-argument callables hold
# the ctypes structs and raw addresses and launch with no per-call Python
# struct building (for tight loops such as a benchmark or a decode loop).
def bind_encode(d: kvq_desc, x: torch.Tensor, tables: Tables, packed: Packed, stream=None):
    from . import lib
    _req(x, "x", (torch.float16,), _kv_shape(d))
    tb, pk, st = tables.struct(), packed.struct(), _stream(stream)
    args = (ctypes.byref(d), x.data_ptr(), ctypes.byref(tb), ctypes.byref(pk), st)
    keep = (d, x, tables, packed, tb, pk)

    def call():
        check(lib.kvq_encode(*args), "kvq_encode")
    call.keep = keep
    return call


def bind_decode(d: kvq_desc, packed: Packed, tables: Tables, out: torch.Tensor, stream=None):
    from . import lib
    _req(out, "out", (torch.float16, torch.float32), _kv_shape(d))
    tb, pk, st = tables.struct(), packed.struct(), _stream(stream)
    fp32 = 1 if out.dtype == torch.float32 else 0
    args = (ctypes.byref(d), ctypes.byref(pk), ctypes.byref(tb), out.data_ptr(), fp32, st)
    keep = (d, packed, tables, out, tb, pk)

    def call():
        check(lib.kvq_decode(*args), "kvq_decode")
    call.keep = keep
    return call


def bind_score(d: kvq_desc, q: torch.Tensor, packed: Packed, tables: Tables, n_tokens: int, scale: float,
               out: torch.Tensor, stream=None, literal: bool = False):
    """A prepared kvq_score call (kvq_score_literal with literal=True)."""
    from . import lib
    hq = _q_heads(d, q)
    _req(out, "scores", (torch.float32,), (d.batch, hq, n_tokens))
    tb, pk, st = tables.struct(), packed.struct(), _stream(stream)
    args = (ctypes.byref(d), q.data_ptr(), hq, ctypes.byref(pk), ctypes.byref(tb), n_tokens,
            ctypes.c_float(scale), out.data_ptr(), st)
    keep = (d, q, packed, tables, out, tb, pk)

    fn, name = (lib.kvq_score_literal, "kvq_score_literal") if literal else (lib.kvq_score, "kvq_score")

    def call():
        check(fn(*args), name)
    call.keep = keep
    return call
