"""A multi-layer model's projections packed on the device.

Every projection is quantized and packed by aq_pack_weights from a device
FP32 weight matrix that a caller-supplied function produces one at a time,
so the FP32 weights of a whole model never sit in memory next to the packed
model (AlignQuant Sec. 3.2: the packed model is what stays resident).
"""

from __future__ import annotations

from contextlib import nullcontext
from dataclasses import dataclass, field

import numpy as np

from .binding import (AQ_PHASE_DECODE, Kv4Cache, PackedExperts, PackedWeights, Rope, aq_attn_kv4, aq_kv4_cache,
                      aq_labels_from_map, aq_linear_decode, aq_linear_prefill, aq_norm_quant, aq_pack_weights,
                      aq_quant_act, aq_rope_kv4, aq_swiglu_quant, aq_workspace_bytes)


@dataclass
class PackedModel:
    """layers[l][name] is the packed projection `name` of layer l."""
    geometry: list            # [(name, N, K)] per layer
    layers: list = field(default_factory=list)

    def nbytes(self) -> int:
        return sum(pw.nbytes() for layer in self.layers for pw in layer.values())

    def __iter__(self):
        for l, layer in enumerate(self.layers):
            for name, _, _ in self.geometry:
                yield l, name, layer[name]


def pack_model(geometry, maps, weight_fn, bN: int = 64, bK: int = 128, progress=None) -> PackedModel:
    """Pack every projection of every layer.

    geometry  : [(name, N, K)], the projections of one layer in call order;
    maps      : maps[l][p] is the [N/bN, K/bK] precision map (4 or 8) of
                projection p of layer l;
    weight_fn : weight_fn(l, name, N, K) -> device FP32 [N, K] weights;
    progress  : optional callable(l) after each layer.
    """
    model = PackedModel(geometry=list(geometry))
    for l, layer_maps in enumerate(maps):
        layer = {}
        for (name, N, K), z in zip(geometry, layer_maps):
            W = weight_fn(l, name, N, K)
            layer[name] = aq_pack_weights(W, aq_labels_from_map(np.asarray(z, dtype=np.uint8)), bN, bK)
            del W
        model.layers.append(layer)
        if progress is not None:
            progress(l)
    return model


@dataclass
class PackedGroup:
    """Projections that share one input, packed as one (App. E.4): the
    members' tile rows are concatenated in member order, so eq. 16's row
    offsets run over the whole group and one quantization of the shared
    input and one linear call serve every member.  members[i] = (name, n0,
    n1): member i owns output features n0 .. n1-1 of the group."""
    packed: PackedWeights
    members: list

    def slices(self, Y) -> dict:
        """The members' outputs: views of the group output Y [M, N]."""
        return {name: Y[:, n0:n1] for name, n0, n1 in self.members}


def pack_group(members, weights, maps, bN: int = 64, bK: int = 128) -> PackedGroup:
    """Pack input-sharing projections as one (App. E.4 grouping).

    members : member names, in the order their rows are concatenated;
    weights : device FP32 [N_i, K] per member (same K, N_i a multiple of bN);
    maps    : [N_i/bN, K/bK] precision maps (4 or 8) per member.
    """
    import torch
    if not members or len(members) != len(weights) or len(weights) != len(maps):
        raise ValueError("one weight matrix and one map per member")
    K = weights[0].shape[1]
    if any(w.shape[1] != K or w.shape[0] % bN for w in weights):
        raise ValueError("members must share K and have whole tile rows")
    spans, n0 = [], 0
    for name, w in zip(members, weights):
        spans.append((name, n0, n0 + w.shape[0]))
        n0 += w.shape[0]
    z = np.concatenate([np.asarray(m, dtype=np.uint8) for m in maps], axis=0)
    W = torch.cat(list(weights), dim=0)
    pw = aq_pack_weights(W, aq_labels_from_map(z), bN, bK)
    del W
    return PackedGroup(packed=pw, members=spans)


def pack_experts(gate, up, down, map_gate_up, map_down, bN: int = 64, bK: int = 128) -> PackedExperts:
    """Pack a mixture-of-experts layer for aq_moe_experts and aq_moe_layer.

    gate, up    : device FP32 [E, I, H];
    down        : device FP32 [E, H, I];
    map_gate_up : [E*2I/bN, H/bK] precision map (4 or 8), the rows of expert e
                  at 2I*e/bN .., its gate rows first;
    map_down    : [E*H/bN, I/bK].
    I and H are multiples of bN and of bK.
    """
    import torch
    if gate.dim() != 3 or up.shape != gate.shape or tuple(down.shape) != (gate.shape[0], gate.shape[2], gate.shape[1]):
        raise ValueError("gate and up must be [E, I, H] and down [E, H, I]")
    E, I, H = gate.shape
    if any(t.dtype != torch.float32 for t in (gate, up, down)):
        raise ValueError("gate, up and down must be float32")
    if I % bN or H % bN or I % bK or H % bK:
        raise ValueError("I and H must be whole tiles")
    for what, z, tiles in (("map_gate_up", map_gate_up, (E * 2 * I // bN, H // bK)), ("map_down", map_down, (E * H // bN, I // bK))):
        if np.shape(z) != tiles:
            raise ValueError(f"{what} must be of shape {tiles}")
    if not gate.is_cuda or up.device != gate.device or down.device != gate.device:
        raise ValueError("gate, up and down must be on one GPU device")
    W = torch.cat([gate, up], dim=1).reshape(E * 2 * I, H).contiguous()
    gu = aq_pack_weights(W, aq_labels_from_map(np.asarray(map_gate_up, dtype=np.uint8)), bN, bK)
    del W
    dn = aq_pack_weights(down.reshape(E * H, I).contiguous(),
                         aq_labels_from_map(np.asarray(map_down, dtype=np.uint8)), bN, bK)
    return PackedExperts(gu, dn, E)


# Rows up to which a projection runs on the decode kernels (a pass over the
# weights per 64 tokens).
DECODE_ROWS = 64


# The arrival counters at the start of a decode workspace, which are zero before its first call.
COUNTER_BYTES = 256 << 10


def _current(device):
    """`device` made current: the projections' calls launch on the current device's stream."""
    import torch
    if device.type != "cuda" or torch.cuda.current_device() == device.index:
        return nullcontext()
    return torch.cuda.device(device)


def linear(pw: PackedWeights, qx, sx, out=None, ws=None):
    """The packed projection of INT8 rows, on the decode or the prefill kernels; ws is
    the decode kernels' workspace (without it that of the stream)."""
    with _current(qx.device):
        if qx.shape[0] <= DECODE_ROWS:
            return aq_linear_decode(pw, qx, sx, out=out, ws=ws)
        return aq_linear_prefill(pw, qx, sx, out=out)


@dataclass
class Decoder:
    """A decoder model on a PackedModel whose layers hold the projections qkv (query
    heads, then key, then value heads), o, gate_up (gate rows, then up rows) and
    down: pre-norm layers with rotary positions, grouped heads, SwiGLU, and a 4-bit cache per
    layer.  The sum with the residual is left to the norm that reads it, so a layer is ten launches
    of this library: norm, qkv, positions and append, attention (with its join), the rows' codes, o, norm,
    gate_up, gate, down.  Query and key heads have no norm of their own.

    Rows behind the last packed sequence (padding: slots of -1) change no other row and come back as anything. Rows that are
    not finite, or that see a cached key or value that is not, come back as NaN."""
    model: PackedModel
    attn_norms: list       # FP32, BF16 or FP16 [H] per layer
    ffn_norms: list
    final_norm: object
    rope: Rope | None
    heads: int             # query heads
    kv_heads: int
    head_dim: int
    eps: float = 1e-6
    _ws_bytes: dict = field(default_factory=dict, init=False, repr=False)   # rows -> bytes of the decode workspace

    def __post_init__(self):
        qkv, o = (self.heads + 2 * self.kv_heads) * self.head_dim, self.heads * self.head_dim
        if not len(self.model.layers) == len(self.attn_norms) == len(self.ffn_norms):
            raise ValueError("one attention norm and one feed-forward norm per layer")
        for layer in self.model.layers:
            H, I = layer["o"].N, layer["down"].K
            shapes = {name: (layer[name].N, layer[name].K) for name in ("qkv", "o", "gate_up", "down")}
            if shapes != {"qkv": (qkv, H), "o": (H, o), "gate_up": (2 * I, H), "down": (H, I)}:
                raise ValueError(f"projections {shapes} do not make a layer of {self.heads} + 2 * {self.kv_heads} heads "
                                 f"of {self.head_dim}")

    def caches(self, pages: int, tokens: int = 64) -> list:
        """An empty cache per layer, `tokens` to a page."""
        return [aq_kv4_cache(pages, tokens, self.kv_heads, self.head_dim, self.model.layers[0]["o"].s8.device)
                for _ in self.model.layers]

    def workspace(self, M: int, device):
        """A workspace of its own for the decode kernels of M rows, None where they need none.  The
        stream's would not do: two graphs captured on one stream would share it, and a call of
        more rows puts a larger one in its place while a graph still holds the old one's address."""
        import torch
        if not 0 < M <= DECODE_ROWS:
            return None
        n = self._ws_bytes.get(M)
        if n is None:
            n = self._ws_bytes[M] = max(aq_workspace_bytes(pw, M, AQ_PHASE_DECODE) for layer in self.model.layers for pw in layer.values())
        if n == 0:
            return None
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        ws[:COUNTER_BYTES].zero_()
        return ws

    def layer(self, l: int, h, delta, cache: Kv4Cache, positions, slots, block_table, kv_len, cu_q=None, ws=None):
        """Layer l on the rows h + delta (delta None: h): (h, delta) of the rows behind
        it, FP32 [M, H]; h is changed in place where delta is given.  ws is a workspace(M) that layers
        one after another share (without it the layer makes its own)."""
        with _current(h.device):
            return self._layer(l, h, delta, cache, positions, slots, block_table, kv_len, cu_q, ws)

    def _layer(self, l, h, delta, cache, positions, slots, block_table, kv_len, cu_q, ws):
        w = self.model.layers[l]
        if ws is None:
            ws = self.workspace(h.shape[0], h.device)
        if delta is None:
            qx, sx = aq_norm_quant(h, self.attn_norms[l], eps=self.eps)
        else:
            qx, sx, h = aq_norm_quant(delta, self.attn_norms[l], residual=h, eps=self.eps, h=h)
        qkv = linear(w["qkv"], qx, sx, ws=ws)
        q = qkv.unflatten(1, (-1, self.head_dim))[:, :self.heads]
        q = aq_rope_kv4(qkv, self.rope, positions, cache, slots, out=q)
        a = aq_attn_kv4(q, cache, block_table, kv_len, cu_q=cu_q)
        o = linear(w["o"], *aq_quant_act(a, mark=True), ws=ws)   # (a row that saw a key or value of NaN stays NaN)
        if delta is None:
            qx, sx, h = aq_norm_quant(o, self.ffn_norms[l], residual=h, eps=self.eps)   # (the caller's rows stay)
        else:
            qx, sx, h = aq_norm_quant(o, self.ffn_norms[l], residual=h, eps=self.eps, h=h)
        qx, sx = aq_swiglu_quant(linear(w["gate_up"], qx, sx, ws=ws))
        return h, linear(w["down"], qx, sx, ws=ws)

    def step(self, x, caches, positions, slots, block_table, kv_len, cu_q=None):
        """All layers, a cache for each, on FP32 rows x [M, H] (a token each: one per sequence
        without cu_q, packed sequences with it): the final norm's INT8 rows and scales, which an
        output projection takes, and the FP32 rows themselves.  The arguments are
        those of aq_rope_kv4 and aq_attn_kv4, kv_len counting these tokens."""
        if len(caches) != len(self.model.layers):
            raise ValueError(f"{len(caches)} caches for {len(self.model.layers)} layers")
        h, delta, ws = x, None, self.workspace(x.shape[0], x.device)
        for l, cache in enumerate(caches):
            h, delta = self.layer(l, h, delta, cache, positions, slots, block_table, kv_len, cu_q, ws)
        return aq_norm_quant(delta, self.final_norm, residual=h, eps=self.eps, h=h)


def tile_row_slices(pw: PackedWeights, tile_rows) -> dict:
    """Host copies of the packed bytes of the given tile rows, concatenated in
    the given order: the W4 and W8 tiles and their scales occupy one
    contiguous run per tile row in each buffer (App. E.1 eq. 16), from
    row_off_b[r] to row_off_b[r + 1]."""
    import torch
    p = pw.plan
    torch.cuda.synchronize()
    off4 = pw.row_off4[:p.offs_bytes].cpu().numpy().view(np.int32)
    off8 = pw.row_off8[:p.offs_bytes].cpu().numpy().view(np.int32)
    t4, t8 = 64 * p.bK // 2, 64 * p.bK     # bytes of one W4 / W8 tile
    out = {k: [] for k in ("w4", "w8", "s4", "s8")}
    for r in tile_rows:
        a4, b4, a8, b8 = int(off4[r]), int(off4[r + 1]), int(off8[r]), int(off8[r + 1])
        out["w4"].append(pw.w4[a4 * t4:b4 * t4].cpu().numpy())
        out["w8"].append(pw.w8[a8 * t8:b8 * t8].cpu().numpy())
        out["s4"].append(pw.s4[a4 * 256:b4 * 256].cpu().numpy().view(np.float32))
        out["s8"].append(pw.s8[a8 * 256:b8 * 256].cpu().numpy().view(np.float32))
    res = {k: np.concatenate(v) if v else np.zeros(0) for k, v in out.items()}
    res["row_off4"], res["row_off8"] = off4, off8
    res["labels"] = pw.labels[:p.labels_bytes].cpu().numpy()
    return res
