"""What is measured of the 8-bit column store's operators.

Three operators, as a decoder layer calls them one after another:

* ``append_q8``  a step's queries and keys rotated, its keys and values written into the 8-bit column
                 store at ``position % rows``; what the blocks that it touches then hold is read back.
* ``unpack_q8``  rows of the store read back as bf16.
* ``attend_q8``  length-aware grouped-query attention over the store.

``run`` computes them with plain torch operations where ``own`` is false, and with the package's
entry points where it is true.

The 8-bit store of K (and of V): codes ``uint8 [cols, Hkv, rows, D]`` and scales ``uint8 [cols, Hkv,
rows / 16]``, one for each block of 16 rows of a head.  Code c under scale byte b stands for
``(c - 128) * 2**(min(b, 29) - 20)``.  A step that writes rows of a block takes the block's new rows (bf16,
at most 65024 in magnitude, NaN as 0) together with the rows that it keeps: those that hold a position
from before the step.  The scale becomes the smallest one that is at least a 127th of their largest
magnitude, and all of them are coded under it, ``128 + rint(x / scale)``.
"""
import math
import random

import torch

own = False

BLOCK = 16      # store rows that share a scale
BIAS = 20       # of the scale byte
TOP = 29        # the largest scale byte in use
LARGEST = 127.0 * 2 ** (TOP - BIAS)
SCALES = [2.0 ** (b - BIAS) for b in range(TOP + 1)]  # (a device's own powers may be off by a bit)


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # --- attention over the store
        # one sequence's token with a short context: what a call costs at least
        dict(name="attend_one_short", kind="attend_q8", S=1, q_min=1, q_max=1, Hq=4, Hkv=1, D=64, rows=256,
             kv_min=200, kv_max=200, causal=1, window=0, drafts=0, pad=0, lens=1),
        # a batch of sequences of every length, one token each
        dict(name="attend_decode", kind="attend_q8", S=32, q_min=1, q_max=1, Hq=16, Hkv=2, D=128, rows=8192,
             kv_min=1, kv_max=8192, causal=1, window=0, drafts=0, pad=0, lens=2),
        # a large batch with long contexts: the store is read at the memory's rate
        dict(name="attend_decode_long", kind="attend_q8", S=64, q_min=1, q_max=1, Hq=32, Hkv=8, D=128, rows=32768,
             kv_min=16384, kv_max=32768, causal=1, window=0, drafts=0, pad=0, lens=3),
        # wide heads, one to three tokens a sequence (a few tokens guessed ahead)
        dict(name="attend_wide_heads", kind="attend_q8", S=13, q_min=1, q_max=3, Hq=16, Hkv=4, D=256, rows=8192,
             kv_min=1000, kv_max=8000, causal=1, window=0, drafts=0, pad=2, lens=4),
        # sliding-window targets of 1 to 16 rows and non-causal 16-row draft blocks on one ring
        dict(name="attend_mixed_ring", kind="attend_q8", S=16, q_min=1, q_max=16, Hq=32, Hkv=8, D=128, rows=4112,
             kv_min=2000, kv_max=60000, causal=1, window=4096, drafts=8, pad=5, lens=5),
        # a chunk of a long prompt behind what is cached of it
        dict(name="attend_chunk", kind="attend_q8", S=1, q_min=1537, q_max=1537, Hq=16, Hkv=2, D=128, rows=32768,
             kv_min=24001, kv_max=24001, causal=1, window=0, drafts=0, pad=0, lens=6),
        # --- a step's keys and values into the store
        # a batch's next tokens
        dict(name="append_decode", kind="append_q8", S=32, q_min=1, q_max=1, Hq=16, Hkv=2, D=128, rows=8192,
             kv_min=1, kv_max=8192, window=0, pad=0, R=128, axes=1, interleaved=0, table=8192, lens=7),
        # a prompt with images: three position axes, padded behind its last row
        dict(name="append_chunk_axes", kind="append_q8", S=1, q_min=4093, q_max=4093, Hq=32, Hkv=8, D=128, rows=8192,
             kv_min=6000, kv_max=6000, window=0, pad=3, R=128, axes=3, interleaved=0, table=8192, lens=8),
        # several prompts' chunks at once into the ring of a sliding-window layer
        dict(name="append_ring_chunks", kind="append_q8", S=5, q_min=100, q_max=1900, Hq=32, Hkv=8, D=128, rows=6144,
             kv_min=2000, kv_max=60000, window=4096, pad=7, R=64, axes=1, interleaved=1, table=65536, lens=9),
        # --- rows of the store read back
        # a batch's last few tokens
        dict(name="unpack_last", kind="unpack_q8", S=16, q_min=1, q_max=16, Hkv=2, D=128, rows=8192,
             kv_min=100, kv_max=8192, window=0, pad=1, lens=10),
        # two whole sequences leave the store (to be kept elsewhere, or read by another kernel)
        dict(name="unpack_sequences", kind="unpack_q8", S=2, q_min=20000, q_max=30000, Hkv=8, D=128, rows=32768,
             kv_min=20000, kv_max=30000, window=0, pad=0, lens=11),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    kind = rng.choice(["attend_q8", "attend_q8", "attend_q8", "append_q8", "append_q8", "unpack_q8"])
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8])
    rows = BLOCK * _log_int(rng, 2, 768)
    long = kind != "attend_q8" or rng.random() < 0.3
    S = _log_int(rng, 1, 8 if long else 64)
    q_max = min(_log_int(rng, 1, 1024 if long else 16), rows // 2)
    q_min = rng.randint(1, q_max)
    window = rng.choice([0, 0, rng.randint(1, rows - q_max + 1)])  # a ring holds the window of a whole step
    kv_max = rows if window == 0 else 4 * rows
    case = dict(kind=kind, S=S, q_min=q_min, q_max=q_max, Hkv=Hkv, D=D, rows=rows, kv_min=rng.randint(1, kv_max),
                kv_max=kv_max, window=window, pad=rng.choice([0, 0, 3]), lens=rng.randrange(1 << 30))
    if kind == "unpack_q8":
        q_max = min(_log_int(rng, 1, 12288), rows)
        return dict(case, q_min=rng.randint(1, q_max), q_max=q_max,
                    window=0 if window == 0 else rng.randint(1, rows - q_max + 1))
    case["Hq"] = Hkv * group
    if kind == "attend_q8":
        case = dict(case, causal=1 if window else rng.randint(0, 1), drafts=0)
        while work(case)["flops"] > 2.5e11:  # no more than the largest listed case
            case["q_max"] = case["q_max"] * 2 // 3
            case["q_min"] = min(case["q_min"], case["q_max"])
        return case
    return dict(case, R=rng.choice([D, D, D // 2, 48]), axes=rng.choice([1, 1, 2, 3]),
                interleaved=rng.randint(0, 1), table=4 * rows + 1)


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


def _read_back(table):
    """The table of the step's rows and of those before them in their first block, and its packed rows."""
    back, t = [], 0
    for _, q_len, col, kv in table:
        n = q_len + (kv - q_len) % BLOCK
        back.append((t, n, col, kv))
        t += n
    return back, t


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


def _filled(case, g):
    """A store in use: codes as normal values have them, blocks' scales a power of two apart or two."""
    shape = (case["S"] + 1, case["Hkv"], case["rows"])
    parts = []
    for _ in range(2):
        codes = torch.empty(shape + (case["D"],), dtype=torch.uint8, device="cuda")
        for col in range(shape[0]):
            n = torch.randn(codes.shape[1:], generator=g, device="cuda")
            codes[col] = n.mul_(30).round_().clamp_(-127, 127).add_(128).to(torch.uint8)
        # 30 steps of 2**-6 to 2**-4: keys and values of order one
        scales = torch.randint(14, 17, (shape[0], shape[1], shape[2] // BLOCK), generator=g, device="cuda",
                               dtype=torch.uint8)
        parts += [codes, scales]
    return parts


def prepare(case, seed):
    g = _generator(seed)
    st = dict(case=case, kind=case["kind"])
    table, modes, T = _segments(case)
    st["T"], st["L"] = T, max(s[1] for s in table)
    st["seq_info"] = torch.tensor(table, dtype=torch.int32, device="cuda")
    if len(set(modes)) > 1:
        st["seg_mode"] = torch.tensor(modes, dtype=torch.int32, device="cuda")
    st["store"] = _filled(case, g)
    if case["kind"] == "unpack_q8":
        return st
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["kind"] == "attend_q8":
        st["q"] = _normal((T, Hq, D), g)
        return st
    # queries, keys and values as one projection leaves them: views of its rows
    qkv = _normal((T, Hq + 2 * Hkv, D), g)
    st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    st["table"] = _rotation_table(case)
    st["sections"] = _sections(case)
    back, st["T_back"] = _read_back(table)
    st["back"] = torch.tensor(back, dtype=torch.int32, device="cuda")
    # one axis: a row's position is its place in its sequence; several: the model gives them
    st["positions"] = None
    if case["axes"] > 1:
        st["positions"] = torch.randint(0, case["table"], (case["axes"], T), generator=g, device="cuda",
                                        dtype=torch.int32)
    return st


# ------------------------------------------------------------------------------- plain forms

def _rotate(x, table, pos, sections, interleaved):
    """x [T, H, D] turned by the angles of pos [axes, T]; the pairs of dims beyond 2 * pairs pass."""
    half = table.shape[1]
    axis = torch.repeat_interleave(torch.arange(len(sections), device=x.device),
                                   torch.tensor(sections, device=x.device), output_size=half)
    cs = table[pos.long()[axis].t(), torch.arange(half, device=x.device)].double()  # [T, half, 2]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    xd = x.double()
    rot, rest = xd[..., :2 * half], xd[..., 2 * half:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
    else:
        a, b = rot[..., :half], rot[..., half:]
    ra, rb = a * cos - b * sin, a * sin + b * cos
    rot = torch.stack([ra, rb], dim=-1).flatten(-2) if interleaved else torch.cat([ra, rb], dim=-1)
    return torch.cat([rot, rest], dim=-1).to(torch.bfloat16)


def _scale(b):
    return torch.tensor(SCALES, device=b.device)[b.long().clamp(max=TOP)]


def _values(codes, scales):
    """What codes [..., rows, D] under scales [..., rows / BLOCK] stand for, in 32 bits (each is exact)."""
    return (codes.float() - 128) * _scale(scales).repeat_interleave(BLOCK, dim=-1)[..., None]


def _scale_byte(amax):
    """The smallest scale that is at least amax / 127."""
    m, e = torch.frexp(amax)                     # amax = m * 2**e, m in [0.5, 1)
    e = e - 7 + (m > 127 / 128).int()            # 127 * 2**e is at least amax
    return torch.where(amax > 0, e + BIAS, torch.zeros_like(e)).clamp(0, TOP)


def _rows_of(seq, T):
    """Each packed row's segment, whether it has one, and its position in the sequence."""
    t = torch.arange(T, device=seq.device)[:, None]
    inside = (t >= seq[:, 0]) & (t < seq[:, 0] + seq[:, 1])  # [T, S]
    seg = inside.int().argmax(1)
    return seg, inside.any(1), seq[seg, 3] - seq[seg, 1] + t[:, 0] - seq[seg, 0]


def _unpack(store, seq, T, rows):
    seg, live, p = _rows_of(seq, T)
    at = live.nonzero()[:, 0]
    col, row = seq[seg[at], 2], p[at] % rows
    out = []
    for codes, scales in (store[:2], store[2:]):
        kept = torch.zeros((T,) + codes.shape[1::2], dtype=torch.bfloat16, device=codes.device)
        v = (codes[col, :, row].float() - 128) * _scale(scales[col, :, row // BLOCK])[..., None]
        kept[at] = v.to(torch.bfloat16)
        out.append(kept)
    return out


def _append(st):
    case, seq, rows = st["case"], st["seq_info"].long(), st["case"]["rows"]
    seg, live, p = _rows_of(seq, st["T"])
    pos = st["positions"] if st["positions"] is not None else p[None]
    # rows of no segment: any position does, nothing of them is kept
    pos = torch.where(live, pos, torch.zeros_like(pos))
    q = _rotate(st["q"], st["table"], pos, st["sections"], case["interleaved"])
    k = _rotate(st["k"], st["table"], pos, st["sections"], case["interleaved"])
    q = torch.where(live[:, None, None], q, torch.zeros_like(q))

    # the blocks that the step writes to, and where in them its rows go
    at = live.nonzero()[:, 0]
    row = p[at] % rows
    blocks, which = torch.unique(seq[seg[at], 2] * (rows // BLOCK) + row // BLOCK, return_inverse=True)
    col, block, slot = blocks // (rows // BLOCK), blocks % (rows // BLOCK), row % BLOCK
    of = torch.empty_like(blocks).index_copy_(0, which, seg[at])
    new = torch.zeros(len(blocks), BLOCK, dtype=torch.bool, device=seq.device)
    new[which, slot] = True
    # the last position before the step in each of a block's rows
    before = (seq[of, 3] - seq[of, 1] - 1)[:, None]
    r = block[:, None] * BLOCK + torch.arange(BLOCK, device=seq.device)
    kept = ~new & (before - torch.remainder(before - r, rows) >= 0)
    use = (new | kept)[:, None, :, None]
    for codes, scales, x in ((*st["store"][:2], k), (*st["store"][2:], st["v"])):
        c = codes.view(codes.shape[0], codes.shape[1], -1, BLOCK, codes.shape[3])
        old = c[col, :, block]                                          # [blocks, Hkv, BLOCK, D]
        v = _values(old, scales[col, :, block][..., None])
        x = x[at].float()
        x = torch.where(x.isnan(), torch.zeros_like(x), x).clamp(-LARGEST, LARGEST)
        v.transpose(1, 2)[which, slot] = x                              # a view: in place
        b = _scale_byte(torch.where(use, v.abs(), torch.zeros_like(v)).amax((-1, -2)))
        n = (torch.round(v / _scale(b)[..., None, None]).clamp(-128, 127) + 128).to(torch.uint8)
        c[col, :, block] = torch.where(use, n, old)
        scales[col, :, block] = b.to(torch.uint8)
    k, v = _unpack(st["store"], st["back"].long(), st["T_back"], rows)
    return dict(q=q, k=k, v=v)


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
    s = q @ _values(kc[col], ks[col]).transpose(-1, -2) / math.sqrt(D)
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
    o = (e.view(S, Hkv, -1, rows) @ _values(vc[col], vs[col])).view(S, Hkv, -1, L, D) / total.clamp_(min=1e-30)
    o = o.permute(0, 3, 1, 2, 4).reshape(S, L, Hq, D).to(torch.bfloat16)
    out = torch.zeros_like(st["q"])
    out[t[inside]] = o[inside]
    return out


def _plain(st):
    if st["kind"] == "unpack_q8":
        k, v = _unpack(st["store"], st["seq_info"].long(), st["T"], st["case"]["rows"])
        return dict(k=k, v=v)
    return _attend(st) if st["kind"] == "attend_q8" else _append(st)


# ------------------------------------------------------------------------- the package's calls

def _calls(st):
    import varlen_gqa_attention_gb300 as pkg

    case = st["case"]
    store = pkg.Q8Store(*st["store"])
    if st["kind"] == "unpack_q8":
        k, v = pkg.sdpa_q8_unpack(store, st["seq_info"], st["T"], window=case["window"])
        return dict(k=k, v=v)
    if st["kind"] == "attend_q8":
        if "workspace" not in st:  # a program keeps one
            need = pkg.q8_workspace_bytes(st["T"], case["Hq"], store, case["S"])
            st["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        return pkg.sdpa_varlen_q8(st["q"], store, st["seq_info"], causal=bool(case["causal"]), window=case["window"],
                                  seg_mode=st.get("seg_mode"), workspace=st["workspace"])
    q = pkg.sdpa_rope_append_q8(st["q"], st["k"], st["v"], store, st["seq_info"], st["table"],
                                positions=st["positions"], sections=st["sections"],
                                interleaved=bool(case["interleaved"]), window=case["window"])
    # what the step's blocks now hold, up to its last row (a window of 1: no row's past counts here)
    k, v = pkg.sdpa_q8_unpack(store, st["back"], st["T_back"], window=1)
    return dict(q=q, k=k, v=v)


def run(state):
    return _calls(state) if own else _plain(state)


# -------------------------------------------------------------------------------------- work

def work(case):
    D, Hkv = case["D"], case["Hkv"]
    table, modes, T = _segments(case)
    live = sum(s[1] for s in table)
    if case["kind"] == "unpack_q8":
        return dict(bytes=2 * live * Hkv * D + 2 * 2 * T * Hkv * D, flops=2 * live * Hkv * D)
    Hq = case["Hq"]
    if case["kind"] == "attend_q8":
        keys = pairs = 0
        for (_, q_len, _, kv), (causal, window) in zip(table, modes):
            first = kv - q_len  # position of the first query row
            lo = max(0, first - window + 1) if window else 0
            keys += kv - lo
            for i in range(q_len):
                hi = first + i + 1 if causal else kv
                pairs += hi - (max(0, first + i - window + 1) if window else 0)
        return dict(bytes=2 * keys * Hkv * D + 2 * keys * Hkv // BLOCK + 2 * (live + T) * Hq * D,
                    flops=4 * D * Hq * pairs)
    _, T_back = _read_back(table)
    read = 2 * live * (Hq + 2 * Hkv) * D + live * case["R"] // 2 * 8
    read += 2 * (T_back - live) * Hkv * D  # what the step's first blocks hold already
    wrote = 2 * T * Hq * D + 2 * live * Hkv * D
    wrote += 2 * T_back * Hkv * D + 2 * 2 * T_back * Hkv * D  # reading the blocks back
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
            y = torch.complex(z[..., u], z[..., w]) * torch.complex(cs[:, 0], cs[:, 1])[:, None]
            z[..., u], z[..., w] = y.real, y.imag
        first += count
    return z


def _decoded(codes, scale_bytes):
    """[..., D] in 64 bits from codes [..., D] and their rows' scale bytes [...]."""
    every = torch.tensor(SCALES, dtype=torch.float64, device="cuda")
    return (codes.double() - 128) * every[scale_bytes.long().clamp(max=TOP)][..., None]


def _written(codes, scales, new, table, rows):
    """The values of the written columns after the step, block by block: {col: [Hkv, rows, D]}."""
    every = torch.tensor(SCALES, dtype=torch.float64, device="cuda")
    out = {}
    for start, n, col, kv in table:
        vals = _decoded(codes[col], scales[col].repeat_interleave(BLOCK, dim=-1))
        first = kv - n
        r = torch.arange(rows, device="cuda")
        holds = first - 1 - (first - 1 - r) % rows >= 0  # rows with a position from before the step
        at = torch.arange(first, kv, device="cuda") % rows
        x = new[start:start + n].double()
        vals[:, at] = torch.nan_to_num(x, nan=0.0).clamp(-LARGEST, LARGEST).transpose(0, 1)
        holds[at] = True
        for b in sorted({int(v) for v in (at // BLOCK).tolist()}):
            here = torch.arange(b * BLOCK, (b + 1) * BLOCK, device="cuda")
            here = here[holds[here]]
            part = vals[:, here]
            most = part.abs().amax((-1, -2))
            fits = (127 * every >= most[:, None])
            s = torch.where(fits.any(-1), every[fits.int().argmax(-1)], every[-1])[:, None, None]
            vals[:, here] = torch.round(part / s).clamp(-128, 127) * s
        out[col] = vals
    return out


def exact(case, seed):
    st = prepare(case, seed)
    table, modes, T = _segments(case)
    Hkv, D, rows = case["Hkv"], case["D"], case["rows"]
    kc, ks, vc, vs = st["store"]
    if case["kind"] == "unpack_q8":
        out = dict(k=torch.zeros(T, Hkv, D, dtype=torch.float64, device="cuda"),
                   v=torch.zeros(T, Hkv, D, dtype=torch.float64, device="cuda"))
        for start, n, col, kv in table:
            at = torch.arange(kv - n, kv, device="cuda") % rows
            for name, codes, scales in (("k", kc, ks), ("v", vc, vs)):
                out[name][start:start + n] = _decoded(codes[col][:, at], scales[col][:, at // BLOCK]).transpose(0, 1)
        return out
    Hq = case["Hq"]
    if case["kind"] == "attend_q8":
        out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
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
            r = at % rows
            for h in range(Hkv):
                k, v = (_decoded(c[col, h, r], b[col, h, r // BLOCK]) for c, b in ((kc, ks), (vc, vs)))
                for hq in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                    w = (st["q"][start:start + n, hq].double() @ k.T * D ** -0.5).masked_fill_(hidden, -math.inf)
                    out[start:start + n, hq] = torch.nan_to_num_(torch.softmax(w, dim=-1)) @ v
        return out
    q = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    keys = torch.zeros(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    for start, n, col, kv in table:
        here = slice(start, start + n)
        pos = st["positions"][:, here] if st["positions"] is not None else torch.arange(kv - n, kv, device="cuda")[None]
        q[here] = _turned(st["q"][here], st, pos)
        # a key has the store's 16 bits before it gets its 8
        keys[here] = _turned(st["k"][here], st, pos).float().to(torch.bfloat16)
    back, T_back = _read_back(table)
    out = dict(q=q)
    for name, codes, scales, new in (("k", kc, ks, keys), ("v", vc, vs, st["v"])):
        cols = _written(codes, scales, new, table, rows)
        out[name] = torch.zeros(T_back, Hkv, D, dtype=torch.float64, device="cuda")
        for start, n, col, kv in back:
            out[name][start:start + n] = cols[col][:, torch.arange(kv - n, kv, device="cuda") % rows].transpose(0, 1)
    return out
