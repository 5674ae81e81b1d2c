"""Measured cases of the operators over a KV cache held in 4 bits.

The cache holds one record of 144 bytes for each (token, KV head): 64 bytes of key codes,
64 of value codes, 4 bf16 key scales, 4 bf16 value scales. A row of 128 channels is four
groups of 32; channel 2i of the row is the low and channel 2i + 1 the high nibble of code
byte i. A nibble n of group g stands for scale[g] * (n - 8). A group's scale is minus an
eighth of its element of largest magnitude (the positive one of a tie counts as smaller), so
that element has the code -8 and the scale is exact in bf16; the codes are
round(x / scale) to the nearest, ties to even, within [-8, 7]. A group whose largest
magnitude is under 2^-100 is held as zeros, and one that has a NaN or an infinity as NaN.
fp32 rows are rounded to bf16 first.

Operators:
  write   new rows of K and V are quantised into the cache at their positions, and what the
          cache then holds for them is read back
  read    the values of a cache, back in rows
  decode  differential attention of one new token for each batch entry over the cache: V2
          (query heads 2p and 2p + 1 are the branches of pair p, over grouped KV heads) and
          V1 (each head has its own K_1 | K_2 and V, an RMSNorm and a scale at the end)
Contiguous caches are [B, L, H, 144]; paged ones a pool [pages, page size, H, 144] with a
block table. Lengths differ from entry to entry.
"""
import math
import random

import torch

own = False

W = 128       # channels of a K or V row
GROUP = 32    # channels of a scale
RECORD = 144  # bytes of a (token, head)
EPS = 1e-5


def listed():
    return [
        # a batch of prompts enters the cache of a V1 layer (sequence 4096, 16 heads)
        dict(name="write_prompt", op="write", B=2, H=16, cap=4096, n_lo=4096, n_hi=4096, page=0,
             packed=False, dtype="bf16", history=False, std=0.125),
        # the new token of every entry of a serving batch: the smallest call, launch latency
        dict(name="write_step", op="write", B=64, H=8, cap=2048, n_lo=1, n_hi=1, page=16,
             packed=False, dtype="bf16", history=True, std=1.0),
        # chunks of odd lengths behind earlier tokens, packed, from an fp32 projection
        dict(name="write_chunks", op="write", B=13, H=8, cap=5000, n_lo=1, n_hi=1531, page=0,
             packed=True, dtype="f32", history=True, std=1.0),
        # a long context back in bf16 rows, for the next chunk's prefill
        dict(name="read_long", op="read", B=1, H=8, cap=65536, n_lo=65536, n_hi=65536, page=64,
             packed=False, dtype="bf16", history=False, std=1.0),
        # a packed batch of ragged contexts in fp32
        dict(name="read_ragged", op="read", B=7, H=2, cap=3001, n_lo=0, n_hi=3001, page=8,
             packed=True, dtype="f32", history=False, std=1.0),
        # one short context: latency
        dict(name="decode_v2_small", op="decode", variant=2, B=1, Hq=16, H=2, cap=600, lo=600, hi=600,
             page=0, std=1.0),
        # a serving batch with lengths of its own for each entry
        dict(name="decode_v2_ragged", op="decode", variant=2, B=24, Hq=64, H=8, cap=8192, lo=1, hi=8191,
             page=0, std=1.0),
        # pages of 16 tokens, 16 query heads over each KV head
        dict(name="decode_v2_paged", op="decode", variant=2, B=32, Hq=32, H=2, cap=16384, lo=500,
             hi=16384, page=16, std=1.0),
        # one very long context: the work is split over its length
        dict(name="decode_v2_long", op="decode", variant=2, B=1, Hq=64, H=8, cap=131072, lo=131072,
             hi=131072, page=0, std=1.0),
        # the decode workload at its full size, the largest call
        dict(name="decode_v2_full", op="decode", variant=2, B=64, Hq=64, H=8, cap=32768, lo=32768,
             hi=32768, page=0, std=1.0),
        # V1, small and paged, with an entry that has no token yet
        dict(name="decode_v1_small", op="decode", variant=1, B=5, Hq=4, H=4, cap=704, lo=0, hi=700,
             page=32, std=0.125),
        # the V1 decode workload at its full size
        dict(name="decode_v1_full", op="decode", variant=1, B=32, Hq=16, H=16, cap=32768, lo=32768,
             hi=32768, page=0, std=0.125),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("write", "read", "decode", "decode", "decode"))
    page = rng.choice((0, 0, 1, 4, 8, 16, 64, 256))
    if op == "decode":
        variant = rng.choice((1, 2, 2))
        H = rng.choice((1, 2, 3, 4, 8, 16))
        group = 1 if variant == 1 else rng.choice((2, 4, 6, 8, 8, 16))
        B = _log(rng, 1, 64)
        cap = _log(rng, 1, max(1, min(131072, 64 * 32768 * 8 // (B * H))))
        hi = rng.randint(max(1, cap // 2), cap)
        lo = rng.choice((0, 1, hi // 2, hi))
        return dict(op=op, variant=variant, B=B, Hq=H * group, H=H, cap=cap, lo=lo, hi=hi, page=page,
                    std=0.125 if variant == 1 else 1.0)
    H = rng.choice((1, 2, 3, 4, 8, 16))
    B = _log(rng, 1, 64)
    cap = _log(rng, 2, max(2, min(65536, 65536 * 8 // (B * H))))
    hi = rng.randint(max(1, cap // 3), max(1, cap // 2) if op == "write" else cap)
    packed = rng.random() < 0.5
    lo = hi if not packed else rng.choice((0, 1, hi // 2))
    return dict(op=op, B=B, H=H, cap=cap, n_lo=lo, n_hi=hi, page=page, packed=packed,
                dtype=rng.choice(("bf16", "f32")), history=op == "write" and rng.random() < 0.5,
                std=rng.choice((0.125, 1.0)))


def _lengths(case, lo, hi):
    """A length for each entry: the longest, the shortest, and others between, by the case alone."""
    r = random.Random("%d %d %d %d" % (case["B"], case["cap"], lo, hi))
    n = [hi, lo] + [r.randint(lo, hi) for _ in range(case["B"])]
    return n[:case["B"]]


def _history(case, lengths):
    """The tokens that each entry holds before a write."""
    if not case["history"]:
        return [0] * case["B"]
    r = random.Random("%d %d" % (case["B"], case["cap"]))
    return [r.randint(0, case["cap"] - n) for n in lengths]


def _grid(lengths):
    """(entry, index within the entry) of every row of a packed batch."""
    entry = [b for b, n in enumerate(lengths) for _ in range(n)]
    index = [i for n in lengths for i in range(n)]
    return entry, index


# ---- the plain form ---------------------------------------------------------------------

def _codes(x):
    """Rows [..., 128] as code bytes [..., 64] and scales [..., 4] (bf16)."""
    x = x.to(torch.bfloat16).float().unflatten(-1, (W // GROUP, GROUP))
    hi, lo = x.amax(-1), x.amin(-1)
    peak = torch.where(hi > -lo, hi, lo)
    s = torch.where(peak.abs() < 2.0 ** -100, torch.zeros_like(peak), peak * -0.125)
    n = torch.round(x / torch.where(s == 0, torch.ones_like(s), s)[..., None]).clamp(-8, 7)
    n = torch.where((s == 0)[..., None], torch.zeros_like(n), n)
    bad = ~torch.isfinite(x).all(-1)
    s = torch.where(bad, torch.full_like(s, math.nan), s)
    n = torch.where(bad[..., None], torch.zeros_like(n), n)
    n = (n + 8).to(torch.uint8).flatten(-2)
    return n[..., 0::2] | (n[..., 1::2] << 4), s.to(torch.bfloat16)


def _records(k, v):
    """K and V rows [..., 128] as cache records [..., 144]."""
    (ck, sk), (cv, sv) = _codes(k), _codes(v)
    return torch.cat((ck, cv, sk.view(torch.uint8), sv.view(torch.uint8)), -1)


def _rows(codes, scales):
    """Code bytes [..., 64] and scale bytes [..., 8] as fp32 rows [..., 128]."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float().sub_(8.0)
    s = scales.contiguous().view(torch.bfloat16).float()
    return n.unflatten(-1, (W // GROUP, GROUP)).mul_(s[..., None]).flatten(-2)


def _k(records):
    return _rows(records[..., :64], records[..., 128:136])


def _v(records):
    return _rows(records[..., 64:128], records[..., 136:144])


def _places(state):
    """(entry, position) of every row of a write or a read, and the same as indices into the cache."""
    if state["cu"] is not None:
        cu = state["cu"].long()
        row = torch.arange(state["total"], device=cu.device)
        entry = torch.searchsorted(cu[1:].contiguous(), row, right=True)
        at = row - cu[entry]
    else:
        entry = torch.arange(state["B"], device=state["cache"].device)[:, None]
        at = torch.arange(state["n"], device=state["cache"].device)[None, :].expand(state["B"], -1)
    at = at + (state["pos"].long()[entry] if state["pos"] is not None else 0)
    if state["table"] is not None:
        page = state["cache"].shape[1]
        return state["table"].long()[entry, at // page], at % page
    return entry, at


def _plain_decode(state):
    cache, q, lam = state["cache"], state["q"].float(), state["lam"]
    B, L = q.shape[0], state["max_kv_len"]
    if state["table"] is not None:
        cache = cache[state["table"].long()].flatten(1, 2)[:, :L]
    H = cache.shape[2]
    hidden = torch.arange(L, device=q.device)[None, :] >= state["kv_len"][:, None]
    if state["variant"] == 1:
        k = _k(cache).unflatten(-1, (2, 64))                       # [B, L, H, 2, 64]
        x = torch.einsum("bhed,blhed->bhel", q, k) * 0.125          # [B, H, 2, L]
    else:
        g = q.unflatten(1, (H, -1))                                # [B, H, group, 128]
        x = torch.einsum("bhed,blhd->bhel", g, _k(cache)) * (1.0 / math.sqrt(128.0))
    x = x.masked_fill(hidden[:, None, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1)
    o = torch.einsum("bhel,blhd->bhed", p, _v(cache).masked_fill(hidden[:, :, None, None], 0.0))
    o = torch.where((total > 0)[..., None], o / total[..., None], torch.zeros_like(o))
    o = o.flatten(1, 2).unflatten(1, (-1, 2))                      # [B, heads or pairs, 2, 128]
    y = o[:, :, 0] - lam[:, None] * o[:, :, 1]
    if state["variant"] == 1:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * (1.0 - state["lambda_init"])
    return y.to(torch.bfloat16)


def _plain(state):
    if state["op"] == "decode":
        return _plain_decode(state)
    places = _places(state)
    if state["op"] == "write":
        state["cache"][places] = _records(state["k"], state["v"])
    records = state["cache"][places]
    return _k(records).to(state["dtype"]), _v(records).to(state["dtype"])


# ---- inputs -----------------------------------------------------------------------------

def _normal(gen, shape, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _filled(gen, lead, H, std):
    """A cache [lead..., H, 144] of quantised normal rows, made in slices of its first axis."""
    cache = torch.empty((*lead, H, RECORD), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 18) // max(1, lead[1] * H))
    for i in range(0, lead[0], step):
        part = cache[i:i + step]
        rows = (*part.shape[:-1], W)
        part.copy_(_records(_normal(gen, rows, std, torch.bfloat16), _normal(gen, rows, std, torch.bfloat16)))
    return cache


def _storage(case, gen):
    """The cache of a case and its block table: pages in a shuffled order, some of them unused."""
    B, H, cap, page = case["B"], case["H"], case["cap"], case["page"]
    if not page:
        return _filled(gen, (B, cap), H, case["std"]), None
    each = (cap + page - 1) // page
    pool = B * each + 3
    table = torch.randperm(pool, generator=gen, device="cuda")[:B * each].view(B, each).int().contiguous()
    return _filled(gen, (pool, page), H, case["std"]), table


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cache, table = _storage(case, gen)
    state = dict(op=case["op"], cache=cache, table=table, max_kv_len=case["cap"], B=case["B"])
    if case["op"] == "decode":
        v1 = case["variant"] == 1
        B, Hq = case["B"], case["Hq"]
        q = _normal(gen, (B, Hq, 2, 64) if v1 else (B, Hq, W), case["std"], torch.bfloat16)
        units = Hq if v1 else Hq // 2
        return state | dict(
            variant=case["variant"], q=q, kv_len=_ints(_lengths(case, case["lo"], case["hi"])),
            lam=0.8 + 0.1 * torch.randn(units, generator=gen, device="cuda"),
            lambda_init=torch.full((1,), 0.777870099559, device="cuda") if v1 else None)
    lengths = _lengths(case, case["n_lo"], case["n_hi"])
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    history = _history(case, lengths)
    total = sum(lengths)
    state |= dict(dtype=dtype, n=case["n_hi"], total=total, pos=_ints(history) if case["history"] else None, cu=None)
    if case["packed"]:
        state["cu"] = _ints([sum(lengths[:i]) for i in range(case["B"] + 1)])
    if case["op"] == "write":
        rows = (total, case["H"], W) if case["packed"] else (case["B"], case["n_hi"], case["H"], W)
        state |= dict(k=_normal(gen, rows, case["std"], dtype), v=_normal(gen, rows, case["std"], dtype))
    return state


def run(state):
    if not own:
        return _plain(state)
    import differential_attention_05_b200 as da
    if state["op"] == "decode":
        return da.diffattn_fwd_decode_kv4(
            state["q"], state["cache"], state["lam"], kv_len=state["kv_len"], lambda_init=state["lambda_init"],
            block_table=state["table"], max_kv_len=state["max_kv_len"], norm_eps=EPS)
    where = dict(pos=state["pos"], cu_seqlens=state["cu"], max_seqlen=state["n"], block_table=state["table"],
                 max_kv_len=state["max_kv_len"])
    if state["op"] == "write":
        da.diffattn_kv4_write(state["k"], state["v"], state["cache"], **where)
    return da.diffattn_kv4_read(state["cache"], n_tokens=state["n"] if state["cu"] is None else state["total"],
                                dtype=state["dtype"], **where)


def work(case):
    """Bytes that have to move and operations of the formulas (a product and a sum are two)."""
    B, H = case["B"], case["H"]
    if case["op"] == "decode":
        keys = sum(_lengths(case, case["lo"], case["hi"]))
        units = case["Hq"] if case["variant"] == 1 else case["Hq"] // 2
        queries = 2 * units
        width = 64 if case["variant"] == 1 else W
        ends = B * (queries * width + units * W) * 2 + 4 * (units + B)
        table = 4 * B * ((case["cap"] + case["page"] - 1) // case["page"]) if case["page"] else 0
        group = queries // H
        return dict(bytes=keys * H * RECORD + ends + table, flops=keys * H * group * 2 * (width + W))
    rows = sum(_lengths(case, case["n_lo"], case["n_hi"])) * H
    row = 2 * W * (2 if case["dtype"] == "bf16" else 4)
    if case["op"] == "read":
        return dict(bytes=rows * (RECORD + row), flops=rows * 2 * W)
    return dict(bytes=rows * (row + RECORD + row), flops=rows * 2 * W * 4)


# ---- the definition in 64 bits ----------------------------------------------------------

def _value_table():
    """[256, 2]: the two codes of a byte."""
    byte = torch.arange(256, dtype=torch.float64, device="cuda")
    high = torch.floor(byte / 16)
    return torch.stack((byte - 16 * high, high), -1) - 8


def _decoded(records, first, scale_at):
    """The rows of a record's codes at byte `first` and scales at byte `scale_at`, in 64 bits."""
    codes = _value_table()[records[..., first:first + 64].long()].reshape(*records.shape[:-1], W)
    bits = records[..., scale_at:scale_at + 8].to(torch.int32)
    scale = ((bits[..., 0::2] + 256 * bits[..., 1::2]) << 16).view(torch.float32).double()
    return codes * scale.repeat_interleave(GROUP, -1)


def _nearest(x):
    """What the cache holds of rows [..., 128], in 64 bits."""
    x = x.to(torch.bfloat16).double()
    out = torch.empty_like(x)
    for g in range(0, W, GROUP):
        part = x[..., g:g + GROUP]
        size = part.abs().amax(-1, keepdim=True)
        negative = (part == -size).any(-1, keepdim=True)
        unit = torch.where(negative, size, -size) / 8
        steps = part / torch.where(size < 2.0 ** -100, torch.ones_like(unit), unit)
        low = torch.floor(steps)
        rest = steps - low
        up = (rest > 0.5) | ((rest == 0.5) & (torch.remainder(low, 2) == 1))
        held = torch.clamp(low + up.double(), -8, 7) * unit
        out[..., g:g + GROUP] = torch.where(size < 2.0 ** -100, torch.zeros_like(held), held)
    return out


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "write":
        return _nearest(state["k"]), _nearest(state["v"])
    cache, table, B = state["cache"], state["table"], case["B"]

    def entry(b, n):
        held = cache[b] if table is None else cache[table[b].long()].flatten(0, 1)
        return held[:n]

    if case["op"] == "read":
        lengths = _lengths(case, case["n_lo"], case["n_hi"])
        held = [entry(b, n) for b, n in enumerate(lengths)]
        held = torch.cat(held) if case["packed"] else torch.stack(held)
        return _decoded(held, 0, 128), _decoded(held, 64, 136)
    out = []
    for b, n in enumerate(_lengths(case, case["lo"], case["hi"])):
        q, lam = state["q"][b].double(), state["lam"].double()
        held = entry(b, n).transpose(0, 1)                          # [H, n, 144]
        k, v = _decoded(held, 0, 128), _decoded(held, 64, 136)
        if case["variant"] == 1:
            x = (k.reshape(k.shape[0], n, 2, 64) * q[:, None]).sum(-1).transpose(1, 2) / 8
        else:
            x = torch.matmul(q.reshape(case["H"], -1, W), k.transpose(1, 2)) / math.sqrt(W)
        o = torch.matmul(torch.softmax(x, -1), v) if n else x.new_zeros((*x.shape[:2], W))
        o = o.reshape(-1, 2, W)
        y = o[:, 0] - lam[:, None] * o[:, 1]
        if case["variant"] == 1:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * (1 - state["lambda_init"].double())
        out.append(y)
    return torch.stack(out)
