"""The latent-attention operators that follow the indexer, as measured cases.

Three operators, over a paged cache of 64-token pages that holds one shared
latent vector a token (512 values) and one rotated key part (64 values):

  store   a token's latent vector and its rotated key part go to their pool
          slot, and the queries' rotary part is rotated in the same call
          (latent_store);
  sparse  attention of every query row over the pool slots that the indexer
          selected for it (sparse_latent_attention);
  paged   attention of every request's rows over the whole of its cached
          tokens (paged_latent_attention).

The pool is bf16 ([pages, 64, 576]) or fp8 (e4m3 codes [pages, 64, 512], a
fp32 scale a token, and the rotated part in bf16).  `run` computes the plain
form, or makes the framework's calls where `own` is true.
"""
import math

import torch

own = False

LATENT, ROPE = 512, 64
DIM = LATENT + ROPE
PAGE = 64
SCALE = 192 ** -0.5  # a query head of 128 + 64 values before it is absorbed
E4M3_MAX = 448.0


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of 64 requests with 4 rows each: latency
        dict(name="store 256 rows bf16", op="store", T=256, H=16, pages=512, maxpos=131072, fp8=False, pad=0, interleaved=True),
        # a prefill chunk with all heads: bandwidth
        dict(name="store 8192 rows fp8", op="store", T=8192, H=64, pages=512, maxpos=131072, fp8=True, pad=0, interleaved=True),
        # an odd batch, its tail padded with tokens that have no slot; rotated by halves
        dict(name="store 777 rows fp8 padded", op="store", T=777, H=20, pages=64, maxpos=40000, fp8=True, pad=41, interleaved=False),
        # one decode token of one request, few heads on this GPU: latency
        dict(name="sparse 1 row", op="sparse", rows=1, H=16, topk=2048, slots=131072, fp8=False, fill="full"),
        # one decode step of 64 requests with 4 rows each, all heads, fp8 cache
        dict(name="sparse 256 rows fp8", op="sparse", rows=256, H=64, topk=2048, slots=262144, fp8=True, fill="full"),
        # a prefill chunk over 35000 keys, all heads
        dict(name="sparse 4096 rows", op="sparse", rows=4096, H=64, topk=2048, slots=35008, fp8=False, fill="full"),
        # a chunk at the start of its requests: rows with few keys or none, odd sizes
        dict(name="sparse 77 rows ragged", op="sparse", rows=77, H=20, topk=515, slots=6400, fp8=False, fill="ragged"),
        # twice the heads, fp8 cache, 64k keys
        dict(name="sparse 1024 rows 128 heads fp8", op="sparse", rows=1024, H=128, topk=2048, slots=65536, fp8=True, fill="full"),
        # one short request, one token: latency
        dict(name="paged 1 x 4096", op="paged", B=1, R=1, H=16, lmin=4096, lmax=4096, fp8=False),
        # decode with 4 rows a request over long contexts: bandwidth
        dict(name="paged 64 x 4, 4096..131072", op="paged", B=64, R=4, H=16, lmin=4096, lmax=131072, fp8=False),
        # odd sizes, one context empty or shorter than its rows, fp8 cache
        dict(name="paged 7 x 3 ragged fp8", op="paged", B=7, R=3, H=20, lmin=0, lmax=5001, fp8=True),
        # single-token decode with 128 heads, fp8 cache
        dict(name="paged 32 x 1, 128 heads fp8", op="paged", B=32, R=1, H=128, lmin=4096, lmax=65536, fp8=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["store", "sparse", "paged"])
    fp8 = rng.random() < 0.5
    if op == "store":
        T = _log_int(rng, 1, 8192)
        return dict(op=op, T=T, H=_log_int(rng, 1, 64), pages=-(-T // PAGE) + rng.randrange(1, 300), maxpos=_log_int(rng, 1000, 131072),
                    fp8=fp8, pad=rng.randrange(0, T) if rng.random() < 0.3 else 0, interleaved=rng.random() < 0.5)
    if op == "sparse":
        rows, H = _log_int(rng, 1, 4096), _log_int(rng, 1, 128)
        if H > 64:
            rows = min(rows, 2048)
        topk = _log_int(rng, 16, 2048)
        return dict(op=op, rows=rows, H=H, topk=topk, slots=PAGE * _log_int(rng, -(-topk // PAGE), 2048), fp8=fp8,
                    fill=rng.choice(["full", "ragged"]))
    B, R, H = _log_int(rng, 1, 64), rng.randrange(1, 9), _log_int(rng, 1, 128)
    most = int(64 * 131072 * 64 / (B * max(64, R * H)))  # the largest listed case's rows x keys
    lmax = _log_int(rng, 1, min(131072, most))
    return dict(op=op, B=B, R=R, H=H, lmin=rng.randrange(0, lmax + 1), lmax=lmax, fp8=fp8)


def _counts(case):
    """Selected keys of each row of a sparse case: all, or from none to all in a fixed pattern."""
    rows, topk = case["rows"], case["topk"]
    return [topk] * rows if case["fill"] == "full" else [topk * ((37 * i) % 101) // 100 for i in range(rows)]


def _lengths(case):
    """Context lengths of a paged case, spread evenly over its range, the longest first."""
    lo, hi = case["lmin"], case["lmax"]
    return [round(lo + (hi - lo) * (1.0 - (0.6180339887498949 * b) % 1.0)) for b in range(case["B"])]


def work(case):
    if case["op"] == "store":
        T, H, stored = case["T"], case["H"], case["T"] - case["pad"]
        token = LATENT + 4 + 2 * ROPE if case["fp8"] else 2 * DIM
        return {"bytes": T * (16 + 4 * ROPE + 2 * H * 2 * ROPE) + stored * (2 * DIM + token),
                "flops": 3 * ROPE * T * (H + 1) + (3 * LATENT * stored if case["fp8"] else 0)}
    token = LATENT + 4 + 2 * ROPE if case["fp8"] else 2 * DIM
    if case["op"] == "sparse":
        n, rows, H = case["slots"], case["rows"], case["H"]
        pairs = sum(_counts(case))
        touched = n * (1.0 - math.prod(1.0 - c / n for c in _counts(case)))
        moved = rows * case["topk"] * 4 + touched * token
    else:
        rows, H, R = case["B"] * case["R"], case["H"], case["R"]
        ls = _lengths(case)
        pairs = sum(max(0, l - R + t + 1) for l in ls for t in range(R))
        moved = sum(ls) * token + 4 * sum(-(-l // PAGE) + 1 for l in ls)
    return {"bytes": moved + rows * H * (2 * DIM + 2 * LATENT + 4), "flops": 2.0 * pairs * H * (DIM + LATENT)}


# ------------------------------------------------------------------ inputs

def _pool(pages, fp8, g):
    """A cache as the store call leaves it: latent vectors whose size differs from token to token."""
    kv = torch.empty(pages, PAGE, DIM, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    size = torch.empty(pages, PAGE, 1, dtype=torch.bfloat16, device="cuda").uniform_(0.6, 1.4, generator=g)
    kv *= size
    if not fp8:
        return dict(kv_pages=kv, s_pages=None, pe_pages=None)
    c, pe = kv[..., :LATENT], kv[..., LATENT:].contiguous()
    s = c.abs().amax(-1).float().clamp_min(1e-4) / E4M3_MAX
    codes = (c / s[..., None]).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return dict(kv_pages=codes, s_pages=s, pe_pages=pe)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    if case["op"] == "store":
        T, H, n = case["T"], case["H"], case["pages"] * PAGE
        # the key projection's output (latent | key part) and the query projection's (128 values | rotary part) as they come
        x = torch.randn(T, DIM, device=dev, generator=g).to(torch.bfloat16)
        qx = torch.randn(T, H, 128 + ROPE, device=dev, generator=g).to(torch.bfloat16)
        q = torch.randn(T, H, DIM, device=dev, generator=g).to(torch.bfloat16)  # absorbed; its last 64 values are written by the call
        inv = 10000.0 ** (-torch.arange(0, ROPE, 2, device=dev, dtype=torch.float64) / ROPE)
        ang = torch.arange(case["maxpos"], device=dev, dtype=torch.float64)[:, None] * inv
        cos_sin = torch.cat([ang.cos(), ang.sin()], -1).float()
        positions = torch.randint(0, case["maxpos"], (T,), device=dev, generator=g)
        slots = torch.randperm(n, device=dev, generator=g)[:T]
        if case["pad"]:
            slots[T - case["pad"]:] = -1
        return dict(case=case, c=x[:, :LATENT], k_pe=x[:, LATENT:], q_pe=qx[..., 128:], q=q, positions=positions, cos_sin=cos_sin, slots=slots,
                    **_pool(case["pages"], case["fp8"], g))
    if case["op"] == "sparse":
        rows, H, topk, n = case["rows"], case["H"], case["topk"], case["slots"]
        q = torch.randn(rows, H, DIM, device=dev, generator=g).to(torch.bfloat16)
        # different slots in any order, as the indexer gives them: rows of a shuffled pool at a step that is prime to its size
        perm = torch.randperm(n, device=dev, generator=g)
        step = 2 * torch.randint(0, n // 2, (rows, 1), device=dev, generator=g) + 1
        step = torch.where(torch.gcd(step, torch.full_like(step, n)) == 1, step, torch.ones_like(step))
        start = torch.randint(0, n, (rows, 1), device=dev, generator=g)
        col = torch.arange(topk, device=dev)
        slots = perm[(start + step * col) % n].to(torch.int32)
        counts = torch.tensor(_counts(case), device=dev)[:, None]
        slots = torch.where(col < counts, slots, -1).contiguous()
        return dict(case=case, q=q, slots=slots, **_pool(n // PAGE, case["fp8"], g))
    B, R, H = case["B"], case["R"], case["H"]
    ls = _lengths(case)
    per = [-(-l // PAGE) for l in ls]
    pages, blocks = max(1, sum(per)), max(1, max(per))
    q = torch.randn(B * R, H, DIM, device=dev, generator=g).to(torch.bfloat16)
    perm = torch.randperm(pages, device=dev, generator=g).to(torch.int32).cpu()
    table, off = torch.full((B, blocks), -1, dtype=torch.int32), 0
    for b, c in enumerate(per):
        table[b, :c] = perm[off:off + c]
        off += c
    return dict(case=case, q=q, block_table=table.to(dev), seq_lens=torch.tensor(ls, dtype=torch.int32, device=dev), R=R, **_pool(pages, case["fp8"], g))


# ------------------------------------------------------------------ one pass

def run(st):
    if own:
        import fp8_mqa_logits_03_b200 as fx
        cache = dict(s_pages=st["s_pages"], pe_pages=st["pe_pages"])
        op = st["case"]["op"]
        if op == "store":
            fx.latent_store(st["c"], st["k_pe"], st["positions"], st["cos_sin"], st["slots"], st["kv_pages"], **cache, q_pe=st["q_pe"],
                            q_out=st["q"][..., LATENT:], interleaved=st["case"]["interleaved"])
            return dict(q=st["q"], kv=st["kv_pages"], s=st["s_pages"], pe=st["pe_pages"])
        if op == "sparse":
            out, lse = fx.sparse_latent_attention(st["q"], st["kv_pages"], st["slots"], SCALE, **cache, return_lse=True)
        else:
            out, lse = fx.paged_latent_attention(st["q"], st["kv_pages"], st["block_table"], st["seq_lens"], st["R"], SCALE, **cache, return_lse=True)
        return dict(out=out, lse=lse)
    return dict(store=_plain_store, sparse=_plain_sparse, paged=_plain_paged)[st["case"]["op"]](st)


def _rotate(x, cos_sin, interleaved):
    x, cos, sin = x.float(), cos_sin[..., : ROPE // 2], cos_sin[..., ROPE // 2:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2).to(torch.bfloat16)
    a, b = x[..., : ROPE // 2], x[..., ROPE // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(torch.bfloat16)


def _plain_store(st):
    cs = st["cos_sin"][st["positions"]]
    inter = st["case"]["interleaved"]
    st["q"][..., LATENT:] = _rotate(st["q_pe"], cs[:, None], inter)
    k_pe = _rotate(st["k_pe"], cs, inter)
    n = st["kv_pages"].shape[0] * PAGE
    kept = (st["slots"] >= 0) & (st["slots"] < n)
    at = st["slots"][kept]
    if not st["case"]["fp8"]:
        st["kv_pages"].view(n, DIM)[at] = torch.cat([st["c"], k_pe], -1)[kept]
    else:
        c = st["c"].float()[kept]
        s = c.abs().amax(-1).clamp_min(1e-4) / E4M3_MAX
        codes = (c / s[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        st["kv_pages"].view(torch.uint8).view(n, LATENT)[at] = codes.view(torch.uint8)
        st["s_pages"].view(n)[at] = s
        st["pe_pages"].view(n, ROPE)[at] = k_pe[kept]
    return dict(q=st["q"], kv=st["kv_pages"], s=st["s_pages"], pe=st["pe_pages"])


def _keys(st, at):
    """The cached keys [..., 576] of pool slots `at`, in 32 bits."""
    kv = st["kv_pages"]
    n = kv.shape[0] * PAGE
    if st["s_pages"] is None:
        return kv.view(n, DIM)[at].float()
    c = kv.view(torch.uint8).view(n, LATENT)[at].view(torch.float8_e4m3fn).float()
    return torch.cat([c * st["s_pages"].view(n)[at][..., None], st["pe_pages"].view(n, ROPE)[at].float()], -1)


def _attend(q, keys, seen):
    """softmax(q k^T) v over the keys that are seen (v: their first 512 values), and the log of the sum; a row that sees none gives 0 and -inf."""
    x = (q.float() @ keys.transpose(-1, -2)).mul_(SCALE).masked_fill_(~seen, float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p @ keys[..., :LATENT]) / torch.where(total == 0, torch.ones_like(total), total)
    return out.to(torch.bfloat16), (top + total.log()).squeeze(-1)


def _plain_sparse(st):
    slots = st["slots"].long()
    out, lse = _attend(st["q"], _keys(st, slots.clamp_min(0)), (slots >= 0)[:, None, :])
    return dict(out=out, lse=lse)


def _plain_paged(st):
    table, R, H = st["block_table"].long().clamp_min(0), st["R"], st["case"]["H"]
    B = table.shape[0]
    at = (table[:, :, None] * PAGE + torch.arange(PAGE, device=table.device)).view(B, -1)
    ends = st["seq_lens"].long()[:, None] - R + 1 + torch.arange(R, device=table.device)
    seen = torch.arange(at.shape[1], device=table.device) < ends[:, :, None]
    out, lse = _attend(st["q"].view(B, R * H, DIM), _keys(st, at), seen.repeat_interleave(H, 1))
    return dict(out=out.view(B * R, H, LATENT), lse=lse.view(B * R, H))


# ------------------------------------------------------------------ in 64 bits

def _exact_code(y):
    """The e4m3 value next to y (half to even), |y| <= 448, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "store":
        half = ROPE // 2
        ang = st["cos_sin"].to(f64)[st["positions"]]
        turn = torch.complex(ang[:, :half], ang[:, half:])

        def rot(x, t):
            x = x.to(f64)
            if case["interleaved"]:
                return torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (half, 2)).contiguous()) * t).flatten(-2)
            y = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * t
            return torch.cat([y.real, y.imag], -1)

        q = st["q"].to(f64)
        q[..., LATENT:] = rot(st["q_pe"], turn[:, None])
        live = case["T"] - case["pad"]
        at, c, pe = st["slots"][:live], st["c"][:live].to(f64), rot(st["k_pe"], turn)[:live]
        kv = st["kv_pages"].to(f64).flatten(0, 1)
        if not case["fp8"]:
            kv[at] = torch.cat([c, pe], -1)
            return dict(q=q, kv=kv.view(-1, PAGE, DIM), s=None, pe=None)
        s, pes = st["s_pages"].to(f64).flatten(), st["pe_pages"].to(f64).flatten(0, 1)
        s[at] = c.abs().amax(-1).clamp_min(1e-4) / E4M3_MAX
        kv[at] = _exact_code(c / s[at][:, None])
        pes[at] = pe
        return dict(q=q, kv=kv.view(-1, PAGE, LATENT), s=s.view(-1, PAGE), pe=pes.view(-1, PAGE, ROPE))
    H = case["H"]
    cache = [st[k].flatten(0, 1) if st[k] is not None else None for k in ("kv_pages", "s_pages", "pe_pages")]

    def keys(at):
        if not case["fp8"]:
            return cache[0][at].to(f64)
        c = cache[0].view(torch.uint8)[at].view(torch.float8_e4m3fn).to(f64)
        return torch.cat([c * cache[1][at].to(f64).unsqueeze(-1), cache[2][at].to(f64)], -1)

    def attend(q, k, dead):
        z = torch.einsum("...hd,...nd->...hn", q.to(f64), k) * SCALE
        z[dead.expand_as(z)] = -math.inf
        lse = torch.logsumexp(z, -1)
        p = torch.exp(z - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None])
        return torch.einsum("...hn,...nd->...hd", p, k[..., :LATENT]), lse

    rows = st["q"].shape[0]
    out = torch.zeros(rows, H, LATENT, dtype=f64, device="cuda")
    lse = torch.full((rows, H), -math.inf, dtype=f64, device="cuda")
    if case["op"] == "sparse":
        for r in range(0, rows, 256):
            s = st["slots"][r:r + 256].long()
            out[r:r + 256], lse[r:r + 256] = attend(st["q"][r:r + 256], keys(s.clamp_min(0)), (s < 0)[:, None, :])
        return dict(out=out, lse=lse)
    for b, l in enumerate(_lengths(case)):
        if l:
            j = torch.arange(l, device="cuda")
            k = keys(st["block_table"][b].long()[j // PAGE] * PAGE + j % PAGE)
            for t in range(case["R"]):
                i = b * case["R"] + t
                out[i], lse[i] = attend(st["q"][i], k, j >= l - case["R"] + t + 1)
    return dict(out=out, lse=lse)
