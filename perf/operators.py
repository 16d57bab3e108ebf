"""Cases of the paged 4-bit key/value cache: the codec (write, read), the
attention that reads it, and the page operations (resize, fork, copy,
compact), each with a plain form in elementary torch operations and with the
calls of the library's binding.

The cache.  A page holds 128 tokens of every key/value head.  For one head of
dimension D it is, in this order,
  key codes    [128 tokens][D channels]    4 bits each
  key scales   [128 tokens][D / 32 groups] 8 bits each
  value codes  [D channels][128 tokens]    4 bits each
  value scales [D / 32 groups][128 tokens] 8 bits each.
A 32-bit word holds eight consecutive codes e0..e7: its nibble i (0..3) is
e[2i] and its nibble 4 + i is e[2i + 1].  The scale of a group of 32 channels
of one token is s = (1 + (c & 7) / 8) * 2^((c >> 3) - 20) for its code c, the
largest magnitude over 7 rounded to the nearest such s; a channel x is held
as round(x / s) + 8 (ties to even).  Values s * (code - 8) are exact in
bfloat16.
"""
import torch

own = False

BLOCK = 128
GROUP = 32
LIMIT = 26880.0  # 7 times the largest scale: larger magnitudes are clamped
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _page_bytes(D):
    return 2 * (BLOCK * D // 2 + BLOCK * D // GROUP)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # One new token over a short cached prompt: the smallest call.
        dict(name="token_short", kind="attn", n=1, Hq=16, Hkv=16, D=128, Lq=1, lo=897, hi=897,
             causal=False, density=0.0, dtype="bf16"),
        # A batch of sequences of very different lengths, shared key heads, one token each.
        dict(name="token_ragged", kind="attn", n=48, Hq=32, Hkv=8, D=128, Lq=1, lo=1, hi=8191,
             causal=False, density=0.0, dtype="bf16"),
        # One token over text, preceding clip and current clip of the 72,000-token scale.
        dict(name="token_long", kind="attn", n=1, Hq=16, Hkv=16, D=128, Lq=1, lo=144512,
             hi=144512, causal=False, density=0.0, dtype="bf16"),
        # A few tokens of every sequence checked at once, in fp32, head dimension 64.
        dict(name="tokens_f32_d64", kind="attn", n=8, Hq=8, Hkv=2, D=64, Lq=4, lo=130, hi=6001,
             causal=True, density=0.0, dtype="f32"),
        # A prompt chunk behind a cached prefix, causal.
        dict(name="chunk_causal", kind="attn", n=3, Hq=16, Hkv=4, D=128, Lq=500, lo=500, hi=4700,
             causal=True, density=0.0, dtype="bf16"),
        # The 8,000-token scale (density 0.625) with its keys in the cache: block lists.
        dict(name="scale_lists", kind="attn", n=1, Hq=16, Hkv=16, D=128, Lq=8000, lo=16512,
             hi=16512, causal=False, density=0.625, dtype="bf16"),
        # The step's new token of every sequence goes into the cache.
        dict(name="write_token", kind="write", n=48, Hkv=8, D=128, T=1, lo=1, hi=8191,
             dtype="bf16"),
        # A finished scale of 18,000 tokens goes into the cache behind the text.
        dict(name="write_scale", kind="write", n=1, Hkv=16, D=128, T=18000, lo=18512, hi=18512,
             dtype="bf16"),
        # A short prefix of some sequences comes back in fp32, head dimension 64.
        dict(name="read_f32_d64", kind="read", n=4, Hkv=8, D=64, T=333, lo=333, hi=1500,
             dtype="f32"),
        # The text and the preceding clip come back as bf16 keys and values for the block front-end.
        dict(name="read_prefix", kind="read", n=1, Hkv=16, D=128, T=41012, lo=41012, hi=41012,
             dtype="bf16"),
        # Eight samples forked from one prompt, each grown by its first token: shared pages,
        # the partial last page copied on the write.
        dict(name="fork_grow", kind="fork", n=8, Hkv=8, D=128, len=4613, others=40),
        # Two full copies of a clip's cache, the first dropped, the pool compacted.
        dict(name="copy_compact", kind="compact", n=2, Hkv=16, D=128, len=41012, others=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["token", "token", "token", "chunk", "lists", "write", "read", "fork",
                       "compact"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    if kind == "token":
        n = _log_int(rng, 1, 64)
        hi = _log_int(rng, 33, max(64, min(144512, 144512 * 16 // (n * Hkv))))
        return dict(kind="attn", n=n, Hq=Hkv * rng.choice([1, 2, 4, 8]), Hkv=Hkv, D=D,
                    Lq=rng.choice([1, 1, 1, 2, 3, 5]), lo=rng.randint(1, hi), hi=hi,
                    causal=rng.random() < 0.5, density=0.0,
                    dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]))
    if kind == "chunk":
        n, Lq = rng.randint(1, 4), _log_int(rng, 12, 1024)
        lo = rng.randint(max(1, Lq // 2), Lq + 500)
        return dict(kind="attn", n=n, Hq=min(16, Hkv * rng.choice([1, 2, 4])), Hkv=Hkv, D=128,
                    Lq=Lq, lo=lo, hi=lo + _log_int(rng, 1, 6000), causal=rng.random() < 0.7,
                    density=0.0, dtype="bf16")
    if kind == "lists":
        Lq = _log_int(rng, 200, 8000)
        L = 512 + Lq + _log_int(rng, 100, 8000)
        return dict(kind="attn", n=1, Hq=Hkv, Hkv=Hkv, D=128, Lq=Lq, lo=L, hi=L, causal=False,
                    density=rng.choice([0.09375, 0.1875, 0.5, 0.625]), dtype="bf16")
    dtype = rng.choice(["bf16", "f32"])
    if kind == "write":
        n, T = rng.randint(1, 48), _log_int(rng, 1, 300)
        if rng.random() < 0.4:
            n, T = 1, _log_int(rng, 300, 9000)
        return dict(kind="write", n=n, Hkv=Hkv, D=D, T=T, lo=T + rng.randint(0, 300),
                    hi=T + 300 + rng.randint(0, 2000), dtype=dtype)
    if kind == "read":
        n, T = rng.randint(1, 8), _log_int(rng, 1, 4000)
        return dict(kind="read", n=n, Hkv=Hkv, D=D, T=T, lo=T, hi=T + rng.randint(1, 2000),
                    dtype=dtype)
    if kind == "fork":
        return dict(kind="fork", n=rng.randint(1, 16), Hkv=Hkv, D=D, len=_log_int(rng, 1, 9000),
                    others=rng.randint(0, 60))
    return dict(kind="compact", n=rng.randint(2, 3), Hkv=Hkv, D=D, len=_log_int(rng, 100, 20000),
                others=0)


def _lens(case):
    """The sequences' lengths: spread from lo to hi, no multiples wanted."""
    n, lo, hi = case["n"], case["lo"], case["hi"]
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * ((7 * i + 3) % n if n % 7 else i) // (n - 1) for i in range(n)]


def work(case):
    H, D = case["Hkv"], case["D"]
    token = 2 * (D // 2 + D // GROUP)  # cache bytes of a token and head
    if case["kind"] == "attn":
        e = 4 if case["dtype"] == "f32" else 2
        rows, Lq = case["Hq"] * case["Lq"], case["Lq"]
        lens = _lens(case)
        if case["density"] > 0:
            _, cnt = _list_sizes(case)
            pairs = case["Hq"] * Lq * min(cnt * BLOCK, lens[0])
        elif case["causal"]:
            pairs = case["Hq"] * sum(max(0, L - Lq + 1 + i) for L in lens for i in range(Lq))
        else:
            pairs = rows * sum(lens)
        return dict(bytes=sum(lens) * H * token + case["n"] * rows * (2 * D * e + 4),
                    flops=4 * pairs * D)
    if case["kind"] in ("write", "read"):
        e = 4 if case["dtype"] == "f32" else 2
        values = case["n"] * case["T"] * H
        # A write case also returns the written tokens as they are held.
        passes = 2 if case["kind"] == "write" else 1
        return dict(bytes=values * (passes * 2 * D * e + token), flops=values * 2 * D * 4)
    pages = -(-case["len"] // BLOCK)
    if case["kind"] == "fork":
        copied = case["n"] if case["len"] % BLOCK else 0
    else:  # n copies of all pages; the last moves into the first one's place
        copied = (case["n"] + 1) * pages
    return dict(bytes=2 * copied * H * _page_bytes(D) + 4 * case["n"] * pages, flops=0)


# ------------------------------------------------------------------ inputs

_LOW, _HIGH = [0, 4, 1, 5], [2, 6, 3, 7]


def _pack(codes):
    """[..., m] codes 0..15 -> [..., m / 2] bytes."""
    w = codes.unflatten(-1, (-1, 8))
    return (w[..., _LOW] | (w[..., _HIGH] << 4)).flatten(-2)


def _unpack(b):
    """[..., m / 2] bytes -> [..., m] codes."""
    w = b.unflatten(-1, (-1, 4))
    return torch.stack([w[..., 0] & 15, w[..., 2] & 15, w[..., 0] >> 4, w[..., 2] >> 4,
                        w[..., 1] & 15, w[..., 3] & 15, w[..., 1] >> 4, w[..., 3] >> 4],
                       -1).flatten(-2)


def _scale(code):
    return ((code.to(torch.int32) + (107 << 3)) << 20).view(torch.float32)


def _quantise(x):
    """[..., D] -> codes [..., D] and scale codes [..., D / 32], uint8.

    The quotients are IEEE divisions (by a tensor: a division by a Python
    number is a product with its reciprocal).  The divisors have at most four
    significant bits, so a rounded quotient is on a border between two codes
    only where the quotient itself is: 32 bits decide as 64 would.
    """
    x = x.float()
    x = torch.where(x == x, x, 0.0).clamp(-LIMIT, LIMIT).unflatten(-1, (-1, GROUP))
    amax = x.abs().amax(-1)
    bits = (amax / torch.full_like(amax, 7.0)).view(torch.int32)
    code = ((bits + 0x7FFFF + ((bits >> 20) & 1)) >> 20) - (107 << 3)
    code = code.clamp(0, 255)
    n = torch.round(x / _scale(code)[..., None]).clamp(-7, 7)
    return (n + 8).to(torch.uint8).flatten(-2), code.to(torch.uint8)


def _join(kc, ks, vc, vs):
    """Codes [..., 128, D] and scale codes [..., 128, D / 32] -> page bytes."""
    return torch.cat([_pack(kc).flatten(-2), ks.flatten(-2),
                      _pack(vc.transpose(-1, -2).contiguous()).flatten(-2),
                      vs.transpose(-1, -2).flatten(-2)], -1)


def _split(page, D):
    a, b = BLOCK * D // 2, BLOCK * D // GROUP
    kb, ks, vb, vs = page.split([a, b, a, b], -1)
    return (_unpack(kb.unflatten(-1, (BLOCK, D // 2))), ks.unflatten(-1, (BLOCK, D // GROUP)),
            _unpack(vb.unflatten(-1, (D, BLOCK // 2))).transpose(-1, -2),
            vs.unflatten(-1, (D // GROUP, BLOCK)).transpose(-1, -2))


def _values(codes, scales):
    x = (codes.float() - 8.0).unflatten(-1, (-1, GROUP))
    return (x * _scale(scales)[..., None]).flatten(-2)


def _list_sizes(case):
    nkb = -(-case["hi"] // BLOCK)
    forced = 4 if nkb > 4 else 0  # the text's blocks
    c = nkb - forced
    return nkb, forced + max(1, -(-int(case["density"] * c * 1000000) // 1000000))


def _tokens(shape, g, spread):
    """Activations: noise around an offset of the 128-token block."""
    x = torch.randn(shape, generator=g, device="cuda")
    blocks = torch.randn(*shape[:-2], -(-shape[-2] // BLOCK), shape[-1], generator=g,
                         device="cuda") * spread
    return x + blocks.repeat_interleave(BLOCK, dim=-2)[..., :shape[-2], :]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind, n, H, D = case["kind"], case["n"], case["Hkv"], case["D"]
    i32 = dict(dtype=torch.int32, device="cuda")
    if kind in ("fork", "compact"):
        return _prepare_pages(case, g)
    lens = _lens(case)
    width = -(-max(lens) // BLOCK)
    counts = [-(-L // BLOCK) for L in lens]
    n_pages = sum(counts) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((n, width), -1, **i32)
    refs = torch.zeros(n_pages, **i32)
    pages = torch.randint(0, 256, (n_pages, H, _page_bytes(D)), generator=g, device="cuda",
                          dtype=torch.uint8)  # what no token was written to is not zero
    at = 0
    for i, c in enumerate(counts):
        ids = order[at:at + c]
        table[i, :c] = ids
        refs[ids.long()] = 1
        at += c
        for h in range(H):
            k = _quantise(_tokens((c, BLOCK, D), g, 0.5))
            v = _quantise(_tokens((c, BLOCK, D), g, 0.0))
            pages[ids.long(), h] = _join(*k, *v)
    s = dict(case=case, pages=pages, refs=refs, table=table, lens=torch.tensor(lens, **i32))
    dt = DTYPES[case["dtype"]]
    if kind == "attn":
        s["q"] = _tokens((n, case["Hq"], case["Lq"], D), g, 0.5).to(dt)
        if case["density"] > 0:
            nkb, cnt = _list_sizes(case)
            nqb = -(-case["Lq"] // BLOCK)
            forced = 4 if nkb > 4 else 0
            score = torch.rand(n, case["Hq"], nqb, nkb, generator=g, device="cuda")
            score[..., :forced] = 2.0
            s["kv_idx"] = score.argsort(-1, descending=True)[..., :cnt].sort(-1)[0].int()
            s["kv_idx"] = s["kv_idx"].contiguous()
            s["kv_cnt"] = torch.full((n, case["Hq"], nqb), cnt, **i32)
    else:
        # The newest T tokens of every sequence are written, or the first T read.
        T = case["T"]
        s["starts"] = s["lens"] - T if kind == "write" else torch.zeros(n, **i32)
        if kind == "write":
            s["k"] = _tokens((n, H, T, D), g, 0.5).to(dt)
            s["v"] = _tokens((n, H, T, D), g, 0.0).to(dt)
        s["k_out"] = torch.zeros(n, H, T, D, device="cuda", dtype=dt)
        s["v_out"] = torch.zeros(n, H, T, D, device="cuda", dtype=dt)
    return s


def _prepare_pages(case, g):
    n, H, D, L = case["n"], case["Hkv"], case["D"], case["len"]
    i32 = dict(dtype=torch.int32, device="cuda")
    count = -(-L // BLOCK)
    live = count + case["others"]
    n_pages = live + n * (count + 1) + 2
    # Sequence 0 is the parent, 1..n its copies, n + 1 holds pages between the parent's.
    table = torch.full((n + 2, max(count + 1, case["others"])), -1, **i32)
    order = torch.randperm(live, generator=g, device="cuda").to(torch.int32)
    table[0, :count] = order[:count]
    table[n + 1, :case["others"]] = order[count:]
    refs = torch.zeros(n_pages, **i32)
    refs[:live] = 1
    lens = torch.tensor([L] + [0] * n + [case["others"] * BLOCK], **i32)
    pages = torch.randint(0, 256, (n_pages, H, _page_bytes(D)), generator=g, device="cuda",
                          dtype=torch.uint8)
    return dict(case=case, pages=pages, refs=refs, table=table, lens=lens,
                src=torch.zeros(n, **i32), dst=torch.arange(1, n + 1, **i32),
                none=torch.zeros(n, **i32), grown=torch.full((n,), L + 1, **i32),
                first=torch.ones(1, **i32), zero=torch.zeros(1, **i32),
                n_live=torch.zeros(1, **i32))


# ------------------------------------------------------------- plain forms

def _plain_attn(s):
    c = s["case"]
    n, Hq, H, D, Lq = c["n"], c["Hq"], c["Hkv"], c["D"], c["Lq"]
    page = s["pages"][s["table"].clamp(min=0).long()].transpose(1, 2)  # [n, H, width, bytes]
    kc, ks, vc, vs = _split(page, D)
    k, v = _values(kc, ks), _values(vc, vs)  # [n, H, width, 128, D]
    width = k.shape[2]
    lens = s["lens"].long()
    pos = torch.arange(width * BLOCK, device="cuda")
    q = s["q"].float() * D ** -0.5
    if c["density"] > 0:
        nqb = s["kv_idx"].shape[2]
        idx = s["kv_idx"].long()
        heads = torch.arange(Hq, device="cuda")[None, :, None, None] // (Hq // H)
        batch = torch.arange(n, device="cuda")[:, None, None, None]
        k = k[batch, heads, idx].flatten(3, 4)  # [n, Hq, nqb, keys, D]
        v = v[batch, heads, idx].flatten(3, 4)
        at = (idx[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten(3, 4)
        pad = nqb * BLOCK - Lq
        q = torch.nn.functional.pad(q, (0, 0, 0, pad)).unflatten(2, (nqb, BLOCK))
        sc = q @ k.transpose(-1, -2)
        sc.masked_fill_((at >= lens[:, None, None, None])[:, :, :, None], float("-inf"))
    else:
        q = q.unflatten(1, (H, Hq // H)).flatten(2, 3)  # [n, H, G * Lq, D]
        sc = q @ k.flatten(2, 3).transpose(-1, -2)
        v = v.flatten(2, 3)
        seen = lens[:, None].expand(n, Lq)
        if c["causal"]:
            seen = seen - (Lq - 1) + torch.arange(Lq, device="cuda")
        seen = seen.repeat(1, Hq // H)[:, None, :, None]
        sc.masked_fill_(pos >= seen, float("-inf"))
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(m == float("-inf"), 0.0, m))
    del sc
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, (p @ v) / total, 0.0)
    lse = (m + torch.log(total))[..., 0]
    if c["density"] > 0:
        out, lse = out.flatten(2, 3)[:, :, :Lq], lse.flatten(2, 3)[:, :, :Lq]
    return out.reshape(n, Hq, Lq, D).to(s["q"].dtype), lse.reshape(n, Hq, Lq).contiguous()


def _touched(s, T):
    """Table columns of the pages that hold T tokens from each start.  A
    sequence that needs one page less repeats its last."""
    start = s["starts"].long()[:, None]
    span = torch.arange((T + 126) // BLOCK + 1, device="cuda")
    return start, torch.minimum(start // BLOCK + span, (start + T - 1) // BLOCK)


def _plain_read(s, T):
    D = s["case"]["D"]
    start, cols = _touched(s, T)
    page = s["pages"][s["table"].gather(1, cols).long()].transpose(1, 2)
    kc, ks, vc, vs = _split(page, D)
    at = start % BLOCK + torch.arange(T, device="cuda")  # [n, T]
    at = at[:, None, :, None].expand(-1, page.shape[1], -1, D)
    k = _values(kc, ks).flatten(2, 3).gather(2, at)
    v = _values(vc, vs).flatten(2, 3).gather(2, at)
    return k.to(s["k_out"].dtype), v.to(s["v_out"].dtype)


def _plain_write(s):
    D, T, H = s["case"]["D"], s["case"]["T"], s["case"]["Hkv"]
    start, cols = _touched(s, T)
    ids = s["table"].gather(1, cols).long()
    old = _split(s["pages"][ids], D)  # [n, pages, H, 128, ...]
    t = cols[..., None] * BLOCK + torch.arange(BLOCK, device="cuda") - start[..., None]
    new = (t >= 0) & (t < T)  # [n, pages, 128]
    at = t.clamp(0, T - 1).flatten(1)[:, None, :, None]

    def merged(old, x):
        x = x.gather(2, at.expand(-1, H, -1, x.shape[-1]))
        x = x.unflatten(2, (-1, BLOCK)).transpose(1, 2)
        return torch.where(new[:, :, None, :, None], x, old)

    fresh = [*_quantise(s["k"]), *_quantise(s["v"])]
    s["pages"][ids] = _join(*(merged(o, x) for o, x in zip(old, fresh)))


def _plain_resize(s, seqs, to):
    table, refs, lens = s["table"], s["refs"], s["lens"]
    seqs, to = seqs.long(), to.long()
    rows, old = table[seqs].long(), lens[seqs].long()
    had, have = (old + 127) // BLOCK, (to + 127) // BLOCK
    grow = to > old
    tail = rows.gather(1, (had - 1).clamp(min=0)[:, None])[:, 0].clamp(min=0)
    fresh = grow & (old % BLOCK > 0) & (refs[tail] > 1)  # a shared partial page is copied
    begin = had - fresh.long()
    need = torch.where(grow, have - begin, 0)
    end = need.cumsum(0)
    fits = end <= (refs == 0).sum()
    free = (refs != 0).int().argsort(stable=True)  # the lowest free pages first
    col = torch.arange(table.shape[1], device="cuda")
    take = (grow & fits)[:, None] & (col >= begin[:, None]) & (col < have[:, None])
    page = free[((end - need)[:, None] + col - begin[:, None]).clamp(0, len(refs) - 1)]
    drop = (col >= have[:, None]) & (col < had[:, None])
    fresh &= fits
    refs.scatter_add_(0, page.flatten(), take.flatten().int())
    refs.scatter_add_(0, rows.clamp(min=0).flatten(), -drop.flatten().int())
    refs.scatter_add_(0, tail, -fresh.int())
    into = page.gather(1, begin.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    s["pages"][torch.where(fresh, into, tail)] = s["pages"][tail]
    table[seqs] = torch.where(take, page, torch.where(drop, -1, rows)).int()
    lens[seqs] = torch.where(fits | ~grow, to, old).int()


def _plain_fork(s, src, dst, deep):
    table, refs, lens = s["table"], s["refs"], s["lens"]
    src, dst = src.long(), dst.long()
    rows = table[src].long()
    count = (lens[src].long() + 127) // BLOCK
    used = torch.arange(table.shape[1], device="cuda") < count[:, None]
    if deep:
        free = (refs != 0).int().argsort(stable=True)
        end = count.cumsum(0)
        rank = (end - count)[:, None] + torch.arange(table.shape[1], device="cuda")
        new = torch.where(used, free[rank.clamp(max=len(refs) - 1)], -1)
        # Every free page takes what it becomes a copy of; the others stay.
        source = torch.arange(len(refs) + 1, device="cuda")
        source[torch.where(used, new, len(refs)).flatten()] = rows.flatten()
        s["pages"].copy_(s["pages"][source[:-1]])
        rows = new
    refs.scatter_add_(0, rows.clamp(min=0).flatten(), used.flatten().int())
    table[dst] = torch.where(used, rows, -1).int()
    lens[dst] = lens[src]


def _plain_compact(s):
    table, refs, lens = s["table"], s["refs"], s["lens"]
    live = refs > 0
    total = live.sum()
    at = torch.arange(len(refs), device="cuda")
    # The k-th live page behind the first `total` goes to the k-th free page among them.
    holes, movers = (~live & (at < total)), (live & (at >= total))
    hole = (~holes).int().argsort(stable=True)
    mover = (~movers).int().argsort(stable=True)
    source = torch.where(holes, mover[(holes.cumsum(0) - 1).clamp(min=0)], at)
    target = torch.where(movers, hole[(movers.cumsum(0) - 1).clamp(min=0)], at)
    s["pages"].copy_(s["pages"][source])
    refs.copy_(torch.where(movers, 0, refs[source]))
    used = torch.arange(table.shape[1], device="cuda") < ((lens.long() + 127) // BLOCK)[:, None]
    table.copy_(torch.where(used, target[table.clamp(min=0).long()].int(), table))
    s["n_live"].copy_(total.int()[None])


# --------------------------------------------------------------------- run

def _cache(s):
    """The handle that a program keeps with its buffers."""
    from block_sparse_attention_18_b200 import sparstar as sp
    if "cache" not in s:
        s["cache"] = sp.Kv4Cache(s["pages"], s["refs"], s["table"], s["lens"], s["case"]["D"])
    return sp, s["cache"]


def run(s):
    c = s["case"]
    kind = c["kind"]
    if own:
        sp, cache = _cache(s)
        if kind == "attn":
            return sp.sparstar_kv4_attn(cache, s["q"], causal=c["causal"],
                                        kv_idx=s.get("kv_idx"), kv_cnt=s.get("kv_cnt"))
        if kind in ("write", "read"):
            if kind == "write":
                sp.sparstar_kv4_write(cache, s["k"], s["v"], starts=s["starts"])
            return sp.sparstar_kv4_read(cache, c["T"], starts=s["starts"], k=s["k_out"],
                                        v=s["v_out"])
        sp.sparstar_kv4_resize(cache, s["none"], seqs=s["dst"])
        if kind == "fork":
            sp.sparstar_kv4_fork(cache, s["src"], s["dst"])
            sp.sparstar_kv4_resize(cache, s["grown"], seqs=s["dst"])
        else:
            sp.sparstar_kv4_fork(cache, s["src"], s["dst"], deep=True)
            sp.sparstar_kv4_resize(cache, s["zero"], seqs=s["first"])
            sp.sparstar_kv4_compact(cache, n_live=s["n_live"])
        return s["pages"], s["refs"], s["table"], s["lens"], s["n_live"]
    if kind == "attn":
        return _plain_attn(s)
    if kind in ("write", "read"):
        if kind == "write":
            _plain_write(s)
        return _plain_read(s, c["T"])
    _plain_resize(s, s["dst"], s["none"])
    if kind == "fork":
        _plain_fork(s, s["src"], s["dst"], False)
        _plain_resize(s, s["dst"], s["grown"])
    else:
        _plain_fork(s, s["src"], s["dst"], True)
        _plain_resize(s, s["first"], s["zero"])
        _plain_compact(s)
    return s["pages"], s["refs"], s["table"], s["lens"], s["n_live"]


# ----------------------------------------------------------- 64-bit values

def _exact_codes(b):
    """Bytes [..., m / 2] -> code - 8 in 64 bits [..., m], code by code."""
    m = 2 * b.shape[-1]
    e = torch.arange(m, device=b.device)
    nibble = (e % 2) * 4 + (e % 8) // 2  # of the element's 32-bit word
    byte = b[..., (e // 8) * 4 + nibble // 2]
    return ((byte >> ((nibble % 2) * 4).to(torch.uint8)) & 15).double() - 8.0


def _exact_scales(c):
    c = c.double()
    e = torch.floor(c / 8)
    return (1 + (c - 8 * e) / 8) * torch.exp2(e - 20)


def _exact_head(s, i, h):
    """Keys and values [len, D] of one sequence and key head, in 64 bits."""
    D, L = s["case"]["D"], int(s["lens"][i])
    page = s["pages"][s["table"][i, :-(-L // BLOCK)].long(), h]
    a, b = BLOCK * D // 2, BLOCK * D // GROUP
    k = _exact_codes(page[:, :a].reshape(-1, D // 2))
    k = k * _exact_scales(page[:, a:a + b].reshape(-1, D // GROUP)).repeat_interleave(GROUP, 1)
    v = _exact_codes(page[:, a + b:2 * a + b].reshape(-1, D, BLOCK // 2))
    sv = _exact_scales(page[:, 2 * a + b:].reshape(-1, D // GROUP, BLOCK))
    v = (v * sv.repeat_interleave(GROUP, 1)).transpose(1, 2).reshape(-1, D)
    return k[:L], v[:L]


def _exact_softmax(x, v):
    """x [..., keys] scores with -inf where masked; outputs and log-sums."""
    m = x.amax(-1, keepdim=True).clamp(min=-1e300)
    w = torch.exp(x - m)
    z = w.sum(-1, keepdim=True)
    return (w @ v) / z.clamp(min=1e-300), (m + torch.log(z))[..., 0]


def _exact_rounded(x):
    """What the cache holds of x [..., D], in 64 bits."""
    x = torch.nan_to_num(x.double(), nan=0.0).clamp(-LIMIT, LIMIT).unflatten(-1, (-1, GROUP))
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True) / torch.tensor(7.0, device=x.device))
    code = ((e.double() - 1 + 20) * 8 + torch.round(m * 16) - 8).clamp(0, 255)
    code = torch.where(m == 0, 0.0, code)
    s = _exact_scales(code)
    return (torch.round(x / s).clamp(-7, 7) * s).flatten(-2)


def exact(case, seed):
    if case["kind"] in ("fork", "compact"):
        return None  # pages are moved, nothing is computed
    s = prepare(case, seed)
    n, H, D = case["n"], case["Hkv"], case["D"]
    if case["kind"] == "write":
        return _exact_rounded(s["k"]), _exact_rounded(s["v"])
    if case["kind"] == "read":
        T = case["T"]
        pairs = [_exact_head(s, i, h) for i in range(n) for h in range(H)]
        return tuple(torch.stack([p[j][:T] for p in pairs]).reshape(n, H, T, D) for j in (0, 1))
    Lq, Hq = case["Lq"], case["Hq"]
    out = torch.zeros(n, Hq, Lq, D, device="cuda", dtype=torch.float64)
    lse = torch.zeros(n, Hq, Lq, device="cuda", dtype=torch.float64)
    for i in range(n):
        L = int(s["lens"][i])
        for h in range(Hq):
            if h % (Hq // H) == 0:
                k, v = _exact_head(s, i, h // (Hq // H))
            q = s["q"][i, h].double() / D ** 0.5
            if case["density"] > 0:
                for b in range(s["kv_idx"].shape[2]):
                    rows = slice(b * BLOCK, min(Lq, (b + 1) * BLOCK))
                    at = s["kv_idx"][i, h, b].long()[:, None] * BLOCK
                    at = (at + torch.arange(BLOCK, device="cuda")).flatten()
                    at = at[at < L]
                    out[i, h, rows], lse[i, h, rows] = _exact_softmax(q[rows] @ k[at].T, v[at])
                continue
            x = q @ k.T
            if case["causal"]:
                last = L - Lq + torch.arange(Lq, device="cuda")
                hidden = torch.arange(L, device="cuda") > last[:, None]
                x.masked_fill_(hidden, float("-inf"))
            out[i, h], lse[i, h] = _exact_softmax(x, v)
    return out, lse
