"""What is measured of the 4-bit column store's operators and of the rotary positions around it.

Four operators, as a decoder layer calls them one after another:

* ``rope``       rotary positions on packed rows ``[T, H, D]``, one position axis or several (time,
                 height, width); with ``inverse`` the gradient of the rotation.
* ``append``     a step's queries and keys rotated, its keys and values written into the bf16 column
                 store at ``position % rows``.
* ``append_q4``  the same into the 4-bit column store.
* ``attend_q4``  length-aware grouped-query attention over the 4-bit column store.

``run`` computes them with plain torch operations where ``own`` is false, and with the package's
entry points where it is true.

The 4-bit store of K (and of V): codes ``uint8 [cols, Hkv, rows, D / 2]`` (byte i: dim 2i in the low
nibble, dim 2i + 1 in the high one) and scales ``uint8 [cols, Hkv, rows, D / 32]``, one per 32 dims.
A nibble c under scale byte b stands for ``(c - 8) * 2**((b >> 3) - 21) * (1 + (b & 7) / 8)``.  A
group is stored from its bf16 values x: the scale nearest to ``max|x| / 7`` (ties to the even byte),
then the codes ``8 + clamp(rint(x / scale), -7, 7)``.
"""
import math
import random

import torch

own = False

GROUP = 32   # dims that share a scale
BIAS = 21    # of the scale byte's exponent


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # --- attention over the 4-bit store
        # one sequence's token with a short context: what a call costs at least
        dict(name="attend_one_short", kind="attend_q4", S=1, q_min=1, q_max=1, Hq=4, Hkv=1, D=64, rows=128,
             kv_min=128, kv_max=128, causal=1, window=0, drafts=0, pad=0, lens=1),
        # a batch of sequences of every length, one token each
        dict(name="attend_decode", kind="attend_q4", S=32, q_min=1, q_max=1, Hq=16, Hkv=2, D=128, rows=8192,
             kv_min=1, kv_max=8192, causal=1, window=0, drafts=0, pad=0, lens=2),
        # a large batch with long contexts: the store is read at the memory's rate
        dict(name="attend_decode_long", kind="attend_q4", S=64, q_min=1, q_max=1, Hq=32, Hkv=8, D=128, rows=32768,
             kv_min=16384, kv_max=32768, causal=1, window=0, drafts=0, pad=0, lens=3),
        # sliding-window targets of 1 to 16 rows and non-causal 16-row draft blocks on one ring
        dict(name="attend_mixed_ring", kind="attend_q4", S=16, q_min=1, q_max=16, Hq=32, Hkv=8, D=128, rows=4112,
             kv_min=2000, kv_max=60000, causal=1, window=4096, drafts=8, pad=5, lens=4),
        # a chunk of a long prompt behind what is cached of it
        dict(name="attend_chunk", kind="attend_q4", S=1, q_min=2048, q_max=2048, Hq=16, Hkv=2, D=128, rows=32768,
             kv_min=32763, kv_max=32763, causal=1, window=0, drafts=0, pad=0, lens=5),
        # --- a step's keys and values into a store
        # a batch's next tokens into the bf16 store
        dict(name="append_decode", kind="append", S=32, q_min=1, q_max=1, Hq=16, Hkv=2, D=128, rows=8192,
             kv_min=1, kv_max=8192, window=0, pad=0, R=128, axes=1, interleaved=0, table=8192, lens=6),
        # a prompt with images: three position axes, padded behind its last row
        dict(name="append_chunk_axes", kind="append", S=1, q_min=4093, q_max=4093, Hq=32, Hkv=8, D=128, rows=8192,
             kv_min=6000, kv_max=6000, window=0, pad=3, R=128, axes=3, interleaved=0, table=8192, lens=7),
        # a batch's next tokens into the 4-bit store
        dict(name="append_q4_decode", kind="append_q4", S=32, q_min=1, q_max=1, Hq=16, Hkv=2, D=128, rows=8192,
             kv_min=1, kv_max=8192, window=0, pad=0, R=128, axes=1, interleaved=0, table=8192, lens=8),
        # several prompts' chunks at once into the 4-bit ring of a sliding-window layer
        dict(name="append_q4_chunks", kind="append_q4", S=5, q_min=100, q_max=1900, Hq=32, Hkv=8, D=128, rows=6144,
             kv_min=2000, kv_max=60000, window=4096, pad=7, R=64, axes=1, interleaved=1, table=65536, lens=9),
        # --- rotary positions on their own
        # one token's heads
        dict(name="rope_one", kind="rope", T=1, H=32, D=128, R=128, axes=1, interleaved=0, inverse=0, table=32768),
        # the patches of a video: time, height and width
        dict(name="rope_video", kind="rope", T=16384, H=16, D=64, R=64, axes=3, interleaved=0, inverse=0, table=4096),
        # the gradient of a partial rotation, pairs side by side, an odd number of rows
        dict(name="rope_gradient", kind="rope", T=4097, H=20, D=256, R=128, axes=1, interleaved=1, inverse=1,
             table=131072),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    kind = rng.choice(["rope", "append", "append_q4", "attend_q4", "attend_q4"])
    D = rng.choice([64, 128, 256])
    R = rng.choice([D, D, D // 2, 48])
    axes = rng.choice([1, 1, 2, 3])
    if kind == "rope":
        return dict(kind=kind, T=_log_int(rng, 1, 16384), H=rng.randint(1, 24), D=D, R=R, axes=axes,
                    interleaved=rng.randint(0, 1), inverse=rng.randint(0, 1), table=_log_int(rng, 64, 100000))
    Hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8])
    rows = 16 * _log_int(rng, 2, 768)
    long = kind != "attend_q4" or rng.random() < 0.3
    S = _log_int(rng, 1, 8 if long else 64)
    q_max = min(_log_int(rng, 1, 1024 if long else 16), rows // 2)
    q_min = rng.randint(1, q_max)
    window = rng.choice([0, 0, rng.randint(1, rows - q_max + 1)])  # a ring holds the window of a whole step
    kv_max = rows if window == 0 else 4 * rows
    case = dict(kind=kind, S=S, q_min=q_min, q_max=q_max, Hq=Hkv * group, Hkv=Hkv, D=D, rows=rows,
                kv_min=rng.randint(1, kv_max), kv_max=kv_max, window=window, pad=rng.choice([0, 0, 3]),
                lens=rng.randrange(1 << 30))
    if kind == "attend_q4":
        case = dict(case, causal=1 if window else rng.randint(0, 1), drafts=0)
        while work(case)["flops"] > 5e11:  # no more than the largest listed case
            case["q_max"] = case["q_max"] * 2 // 3
            case["q_min"] = min(case["q_min"], case["q_max"])
        return case
    return dict(case, R=R, axes=axes, interleaved=rng.randint(0, 1), table=4 * rows + 1)


def _segments(case):
    """The step's segment table on the host: (q_start, q_len, col, kv_end), (causal, window) of each
    segment, and the packed rows with the padding behind them.  A case's lengths are its own, not
    its inputs' seed's, so that its work is known from the case."""
    rng = random.Random(case["lens"])
    S, rows = case["S"], case["rows"]
    cols = rng.sample(range(S + 1), S)  # one column stays free
    table, modes, t = [], [], 0
    for s in range(S):
        q_len = rng.randint(case["q_min"], case["q_max"])
        kv = max(q_len, rng.randint(case["kv_min"], case["kv_max"]))
        causal, window = case.get("causal", 1), case["window"]
        if s >= S - case.get("drafts", 0):  # a draft block: every row of it sees the whole context
            q_len, causal, window = 16, 0, 0
            kv = rng.randint(16, rows)
        table.append((t, q_len, cols[s], kv))
        modes.append((causal, window))
        t += q_len
    return table, modes, t + case["pad"]


def _sections(case):
    """Rotated pairs of each position axis: the first gets what the others leave."""
    half, axes = case["R"] // 2, case["axes"]
    each = half // axes
    return (half - each * (axes - 1),) + (each,) * (axes - 1)


# ------------------------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _rotation_table(case):
    """cos and sin of position p times the frequency of pair j, [positions, R / 2, 2], from 64 bits."""
    half = case["R"] // 2
    freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    angle = torch.arange(case["table"], device="cuda", dtype=torch.float64)[:, None] * freq
    return torch.stack([torch.cos(angle), torch.sin(angle)], dim=-1).float()


def _axes_positions(case, T, g):
    return torch.randint(0, case["table"], (case["axes"], T), generator=g, device="cuda", dtype=torch.int32)


def _filled_q4(case, g):
    """A store in use: codes as normal values have them, scales spread over a few powers of two."""
    shape = (case["S"] + 1, case["Hkv"], case["rows"])
    parts = []
    for _ in range(2):
        codes = torch.empty(shape + (case["D"] // 2,), dtype=torch.uint8, device="cuda")
        for col in range(shape[0]):
            n = torch.randn((2,) + codes.shape[1:], generator=g, device="cuda").mul_(2.6).round_().clamp_(-7, 7).add_(8)
            codes[col] = (n[0] + 16 * n[1]).to(torch.uint8)
        # 0.2 to 0.6 around: keys and values of order one
        scales = torch.randint(142, 158, shape + (case["D"] // GROUP,), generator=g, device="cuda", dtype=torch.uint8)
        parts += [codes, scales]
    return parts


def prepare(case, seed):
    g = _generator(seed)
    st = dict(case=case, kind=case["kind"])
    if case["kind"] == "rope":
        st["x"] = _normal((case["T"], case["H"], case["D"]), g)
        st["table"] = _rotation_table(case)
        st["positions"] = _axes_positions(case, case["T"], g)
        st["sections"] = _sections(case)
        return st
    table, modes, T = _segments(case)
    st["T"], st["L"] = T, max(s[1] for s in table)
    st["seq_info"] = torch.tensor(table, dtype=torch.int32, device="cuda")
    if len(set(modes)) > 1:
        st["seg_mode"] = torch.tensor(modes, dtype=torch.int32, device="cuda")
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["kind"] == "attend_q4":
        st["q"] = _normal((T, Hq, D), g)
        st["store"] = _filled_q4(case, g)
        return st
    # queries, keys and values as one projection leaves them: views of its rows
    qkv = _normal((T, Hq + 2 * Hkv, D), g)
    st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    st["table"] = _rotation_table(case)
    st["sections"] = _sections(case)
    # one axis: a row's position is its place in its sequence; several: the model gives them
    st["positions"] = _axes_positions(case, T, g) if case["axes"] > 1 else None
    if case["kind"] == "append":
        shape = (case["rows"], case["S"] + 1, Hkv, D)
        st["k_store"], st["v_store"] = _normal(shape, g), _normal(shape, g)
    else:
        st["store"] = _filled_q4(case, g)
    return st


# ------------------------------------------------------------------------------- plain forms

def _rotate(x, table, pos, sections, interleaved, inverse=False):
    """x [T, H, D] turned by the angles of pos [axes, T]; the pairs of dims beyond 2 * pairs pass."""
    half = table.shape[1]
    axis = torch.repeat_interleave(torch.arange(len(sections), device=x.device),
                                   torch.tensor(sections, device=x.device), output_size=half)
    cs = table[pos.long()[axis].t(), torch.arange(half, device=x.device)].double()  # [T, half, 2]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    if inverse:
        sin = -sin
    xd = x.double()
    rot, rest = xd[..., :2 * half], xd[..., 2 * half:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
    else:
        a, b = rot[..., :half], rot[..., half:]
    ra, rb = a * cos - b * sin, a * sin + b * cos
    rot = torch.stack([ra, rb], dim=-1).flatten(-2) if interleaved else torch.cat([ra, rb], dim=-1)
    return torch.cat([rot, rest], dim=-1).to(torch.bfloat16)


def _q4_values(codes, scales):
    """What the codes stand for, [..., D] in 32 bits (each value is exact)."""
    n = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).float() - 8
    b = scales.int()
    s = torch.ldexp(1 + (b & 7).float() / 8, (b >> 3) - BIAS)
    return n * s.repeat_interleave(GROUP, dim=-1)


def _q4_pack(x):
    """bf16 [..., D] to (codes, scales)."""
    v = x.float().unflatten(-1, (-1, GROUP))
    m, e = torch.frexp(v.abs().amax(-1) / 7)       # m in [0.5, 1)
    steps = torch.round(m * 16)                    # 8 to 16 eighths, ties to even
    b = torch.where(m > 0, steps.int() - 8 + 8 * (e - 1 + BIAS), torch.zeros_like(e)).clamp(0, 255)
    s = torch.ldexp(1 + (b & 7).float() / 8, (b >> 3) - BIAS)
    n = (torch.round(v / s[..., None]).clamp(-7, 7) + 8).to(torch.uint8).flatten(-2)
    return n[..., 0::2] | (n[..., 1::2] << 4), b.to(torch.uint8)


def _rows_of(st):
    """Each packed row's segment, whether it has one, and its position in the sequence."""
    seq = st["seq_info"].long()
    t = torch.arange(st["T"], device=seq.device)[:, None]
    inside = (t >= seq[:, 0]) & (t < seq[:, 0] + seq[:, 1])  # [T, S]
    seg = inside.int().argmax(1)
    return seg, inside.any(1), seq[seg, 3] - seq[seg, 1] + t[:, 0] - seq[seg, 0]


def _append(st):
    seg, live, p = _rows_of(st)
    case = st["case"]
    pos = st["positions"] if st["positions"] is not None else p[None]
    # rows of no segment: any position does, nothing of them is kept
    pos = torch.where(live, pos, torch.zeros_like(pos))
    q = _rotate(st["q"], st["table"], pos, st["sections"], case["interleaved"])
    k = _rotate(st["k"], st["table"], pos, st["sections"], case["interleaved"])
    q = torch.where(live[:, None, None], q, torch.zeros_like(q))
    at = live.nonzero()[:, 0]
    col, row = st["seq_info"].long()[seg[at], 2], p[at] % case["rows"]
    if case["kind"] == "append":
        st["k_store"][row, col] = k[at]
        st["v_store"][row, col] = st["v"][at]
        return dict(q=q, k_store=st["k_store"], v_store=st["v_store"])
    kc, ks, vc, vs = st["store"]
    kept = []
    for codes, scales, new in ((kc, ks, k), (vc, vs, st["v"])):  # K, then V
        c, b = _q4_pack(new[at])
        codes[col, :, row], scales[col, :, row] = c, b
        rows = torch.zeros_like(new)
        rows[at] = _q4_values(codes[col, :, row], scales[col, :, row]).to(torch.bfloat16)
        kept.append(rows)
    return dict(q=q, k=kept[0], v=kept[1])


def _attend(st):
    case, seq, T, L = st["case"], st["seq_info"].long(), st["T"], st["L"]
    Hq, Hkv, D, rows, S = case["Hq"], case["Hkv"], case["D"], case["rows"], case["S"]
    i = torch.arange(L, device=seq.device)
    inside = i < seq[:, 1:2]                                            # [S, L]
    t = seq[:, 0:1] + i
    q = st["q"][t.clamp(max=T - 1)].float().view(S, L, Hkv, Hq // Hkv, D)
    q = q.permute(0, 2, 3, 1, 4).reshape(S, Hkv, -1, D)                 # rows: (head of the group, i)
    kc, ks, vc, vs = st["store"]
    col = seq[:, 2]
    s = q @ _q4_values(kc[col], ks[col]).transpose(-1, -2) / math.sqrt(D)
    # store row r holds the last position below kv_end that is r modulo the rows
    r = torch.arange(rows, device=seq.device)
    j = seq[:, 3:4] - 1 - torch.remainder(seq[:, 3:4] - 1 - r, rows)    # [S, rows]
    p = (seq[:, 3:4] - seq[:, 1:2] + i)[:, :, None]                     # [S, L, 1]
    if "seg_mode" in st:
        causal, window = st["seg_mode"].long()[:, 0, None, None], st["seg_mode"].long()[:, 1, None, None]
    else:
        causal, window = torch.tensor(case["causal"], device=seq.device), torch.tensor(case["window"], device=seq.device)
    j = j[:, None, :]
    seen = (j >= 0) & ((causal == 0) | (j <= p)) & ((window <= 0) | (j > p - window))
    s = s.view(S, Hkv, Hq // Hkv, L, rows).masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp_(min=-3e38)                      # a row that sees nothing: no inf - inf
    e = s.sub_(m).exp_()
    total = e.sum(-1, keepdim=True)
    o = (e.view(S, Hkv, -1, rows) @ _q4_values(vc[col], vs[col])).view(S, Hkv, -1, L, D) / total.clamp_(min=1e-30)
    o = o.permute(0, 3, 1, 2, 4).reshape(S, L, Hq, D).to(torch.bfloat16)
    out = torch.zeros_like(st["q"])
    out[t[inside]] = o[inside]
    return out


def _plain(st):
    if st["kind"] == "rope":
        case = st["case"]
        return _rotate(st["x"], st["table"], st["positions"], st["sections"], case["interleaved"], case["inverse"])
    return _attend(st) if st["kind"] == "attend_q4" else _append(st)


# ------------------------------------------------------------------------- the package's calls

def _calls(st):
    import varlen_gqa_attention_gb300 as pkg

    case = st["case"]
    if st["kind"] == "rope":
        return pkg.sdpa_rope(st["x"], st["table"], st["positions"], sections=st["sections"],
                             interleaved=bool(case["interleaved"]), inverse=bool(case["inverse"]))
    if st["kind"] == "attend_q4":
        store = pkg.Q4Store(*st["store"])
        if "workspace" not in st:  # a program keeps one
            need = pkg.q4_workspace_bytes(st["T"], case["Hq"], store, case["S"])
            st["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        return pkg.sdpa_varlen_q4(st["q"], store, st["seq_info"], causal=bool(case["causal"]), window=case["window"],
                                  seg_mode=st.get("seg_mode"), workspace=st["workspace"])
    how = dict(positions=st["positions"], sections=st["sections"], interleaved=bool(case["interleaved"]),
               window=case["window"])
    if st["kind"] == "append":
        q = pkg.sdpa_rope_append(st["q"], st["k"], st["v"], st["k_store"], st["v_store"], st["seq_info"], st["table"],
                                 **how)
        return dict(q=q, k_store=st["k_store"], v_store=st["v_store"])
    store = pkg.Q4Store(*st["store"])
    q = pkg.sdpa_rope_append_q4(st["q"], st["k"], st["v"], store, st["seq_info"], st["table"], **how)
    # the step's rows as the store now has them
    k, v = pkg.sdpa_q4_unpack(store, st["seq_info"], st["T"], window=case["window"])
    return dict(q=q, k=k, v=v)


def run(state):
    return _calls(state) if own else _plain(state)


# -------------------------------------------------------------------------------------- work

def work(case):
    D = case["D"]
    if case["kind"] == "rope":
        n = case["T"] * case["H"] * D
        # the table's rows that the positions name: each once
        angles = min(case["T"] * case["axes"], case["table"]) * case["R"] // 2 // case["axes"] * 8
        return dict(bytes=4 * n + angles + 4 * case["T"] * case["axes"], flops=3 * case["T"] * case["H"] * case["R"])
    table, modes, T = _segments(case)
    Hq, Hkv, live = case["Hq"], case["Hkv"], sum(s[1] for s in table)
    row_q4 = D // 2 + D // GROUP
    if case["kind"] == "attend_q4":
        keys = pairs = 0
        for (_, q_len, _, kv), (causal, window) in zip(table, modes):
            first = kv - q_len  # position of the first query row
            lo = max(0, first - window + 1) if window else 0
            keys += kv - lo
            for i in range(q_len):
                hi = first + i + 1 if causal else kv
                pairs += hi - (max(0, first + i - window + 1) if window else 0)
        return dict(bytes=2 * keys * Hkv * row_q4 + 2 * (live + T) * Hq * D, flops=4 * D * Hq * pairs)
    read = 2 * live * (Hq + 2 * Hkv) * D + live * case["R"] // 2 * 8
    wrote = 2 * T * Hq * D + 2 * live * Hkv * (2 * D if case["kind"] == "append" else row_q4)
    if case["kind"] == "append_q4":  # reading the step's rows back
        wrote += 2 * live * Hkv * row_q4 + 2 * 2 * T * Hkv * D
    return dict(bytes=read + wrote, flops=3 * live * (Hq + Hkv) * case["R"])


# ---------------------------------------------------------------------- the definition, 64 bits

def _turned(x, st, pos):
    """x [n, H, D] in 64 bits as complex numbers, pair by pair, times e^(i angle)."""
    case, table = st["case"], st["table"].double()
    half = case["R"] // 2
    z = x.double().clone()
    first = 0
    for a, count in enumerate(st["sections"]):
        for jp in range(first, first + count):
            u, w = (2 * jp, 2 * jp + 1) if case["interleaved"] else (jp, jp + half)
            cs = table[pos[a].long(), jp]
            turn = torch.complex(cs[:, 0], -cs[:, 1] if case.get("inverse") else cs[:, 1])
            y = torch.complex(z[..., u], z[..., w]) * turn[:, None]
            z[..., u], z[..., w] = y.real, y.imag
        first += count
    return z


def _nearest_q4(x):
    """The values that the store has for bf16 x [..., D], by search over the 256 scales."""
    x = x.double()
    all_s = torch.tensor([2.0 ** ((b >> 3) - BIAS) * (1 + (b & 7) / 8) for b in range(256)], dtype=torch.float64,
                         device=x.device)
    out = torch.empty_like(x)
    for g0 in range(0, x.shape[-1], GROUP):
        part = x[..., g0:g0 + GROUP]
        want = (part.abs().amax(-1).float() / 7).double()
        up = torch.searchsorted(all_s, want).clamp(1, 255)  # first scale that is not below
        above, below = all_s[up] - want, want - all_s[up - 1]
        b = torch.where((above < below) | ((above == below) & (up % 2 == 0)), up, up - 1)
        s = all_s[b][..., None]
        out[..., g0:g0 + GROUP] = torch.round(part / s).clamp(-7, 7) * s
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "rope":
        return _turned(st["x"], st, st["positions"])
    table, modes, T = _segments(case)
    Hq, Hkv, D, rows = case["Hq"], case["Hkv"], case["D"], case["rows"]
    if case["kind"] == "attend_q4":
        out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
        kc, ks, vc, vs = st["store"]
        for (start, n, col, kv), (causal, window) in zip(table, modes):
            first = kv - n
            lo = max(0, first - window + 1) if window else 0
            at = torch.arange(lo, kv, device="cuda")
            p = torch.arange(first, kv, device="cuda")[:, None]
            hidden = torch.zeros(n, kv - lo, dtype=torch.bool, device="cuda")
            if causal:
                hidden |= at > p
            if window:
                hidden |= at <= p - window
            for h in range(Hkv):
                k, v = (_decoded(c[col, h, at % rows], b[col, h, at % rows]) for c, b in ((kc, ks), (vc, vs)))
                for hq in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                    w = (st["q"][start:start + n, hq].double() @ k.T * D ** -0.5).masked_fill_(hidden, -math.inf)
                    out[start:start + n, hq] = torch.nan_to_num_(torch.softmax(w, dim=-1)) @ v
        return out
    q = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    kept = torch.zeros(2, T, Hkv, D, dtype=torch.float64, device="cuda")
    stores = [st["k_store"].double(), st["v_store"].double()] if case["kind"] == "append" else None
    for start, n, col, kv in table:
        here = slice(start, start + n)
        p = torch.arange(kv - n, kv, device="cuda")
        pos = st["positions"][:, here] if st["positions"] is not None else p[None]
        q[here] = _turned(st["q"][here], st, pos)
        k, v = _turned(st["k"][here], st, pos), st["v"][here].double()
        if stores:
            stores[0][p % rows, col], stores[1][p % rows, col] = k, v
        else:  # a key has the store's 16 bits before it gets its 4
            kept[0, here], kept[1, here] = _nearest_q4(k.float().to(torch.bfloat16)), _nearest_q4(v)
    return dict(q=q, k_store=stores[0], v_store=stores[1]) if stores else dict(q=q, k=kept[0], v=kept[1])


def _decoded(codes, scales):
    """[n, D] in 64 bits from bytes [n, D / 2] and [n, D / 32], byte by byte."""
    v = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    v[:, 0::2] = codes.double() % 16 - 8
    v[:, 1::2] = torch.div(codes.double(), 16, rounding_mode="floor") - 8
    scale = 2.0 ** (torch.div(scales.double(), 8, rounding_mode="floor") - BIAS) * (1 + scales.double() % 8 / 8)
    for g in range(scales.shape[1]):
        v[:, GROUP * g:GROUP * (g + 1)] *= scale[:, g:g + 1]
    return v
