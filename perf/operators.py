"""Cases of the framework's packed attention and 4-bit projection operators, with their plain forms.

Three operators, as a transformer layer served in 4 bits meets them:

  quantize   rows of activations or weights to microscaled 4-bit floating point (e2m1 elements,
             one power-of-two scale for each 32 of a row), given back as the values they stand for
  linear     y = a W^T + bias: a quantised on the way in, W held in 4 bits, fp32 sums
  attention  softmax attention over packed sequences of different lengths: grouped heads, causal
             or not, the queries being the last rows of their sequence (a whole prompt, a chunk of
             one behind its prefix, or single tokens over a cache); out and the log-sum-exp

Microscaling (OCP MX v1.0, FP4): for each block of 32, e = clamp(floor(log2 max|x|) - 2, -127, 127),
each element x / 2^e rounded to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to the even code),
saturating at 6.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 32
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one token's hidden row of a 12 x 128-head model: latency alone
        {"name": "quantize_token", "op": "quantize", "rows": 1, "k": 1536, "dtype": "bf16"},
        # odd rows, a row length that is no multiple of 128, fp32 input (a checkpoint's weight)
        {"name": "quantize_ragged_f32", "op": "quantize", "rows": 2711, "k": 4128, "dtype": "f32"},
        # a whole window of 8 blocks x 6240 tokens
        {"name": "quantize_window", "op": "quantize", "rows": 49920, "k": 1536, "dtype": "bf16"},
        # single-token decoding: bound by the 4-bit weights
        {"name": "linear_token", "op": "linear", "m": 1, "n": 4096, "k": 4096, "bias": False, "dtype": "bf16"},
        # a small batch of tokens, fp32 out (a head's logits)
        {"name": "linear_batch", "op": "linear", "m": 19, "n": 6144, "k": 2048, "bias": True, "dtype": "f32"},
        # a short packed prompt batch, q/k/v width of the 12 x 128-head model
        {"name": "linear_prompt", "op": "linear", "m": 333, "n": 4608, "k": 1536, "bias": True, "dtype": "f16"},
        # a window of 4 blocks x 12480/4 tokens into a wide feed-forward: bound by the tensor cores
        {"name": "linear_window", "op": "linear", "m": 12480, "n": 11008, "k": 4096, "bias": True, "dtype": "bf16"},
        # one short prompt, one head per k/v head
        {"name": "attention_short", "op": "attention", "heads": 12, "kv_heads": 12, "head_dim": 64, "dtype": "f16",
         "q_lens": "77", "k_lens": "77", "capacity": 0, "causal": True},
        # decoding: one token for each of 8 sequences over padded caches
        {"name": "attention_decode", "op": "attention", "heads": 32, "kv_heads": 8, "head_dim": 128, "dtype": "bf16",
         "q_lens": "1,1,1,1,1,1,1,1", "k_lens": "8191,1,5000,3333,7168,129,6240,4097", "capacity": 8192,
         "causal": True},
        # prompts of several lengths packed together
        {"name": "attention_packed", "op": "attention", "heads": 32, "kv_heads": 8, "head_dim": 128, "dtype": "bf16",
         "q_lens": "1350,1,777,2048,0,130,1999,512,63", "k_lens": "1350,1,777,2048,0,130,1999,512,63",
         "capacity": 0, "causal": True},
        # chunks of prompts behind a prefix; the last sequence has more queries than keys: rows that see nothing
        {"name": "attention_chunks", "op": "attention", "heads": 24, "kv_heads": 8, "head_dim": 64, "dtype": "f16",
         "q_lens": "512,257,1000,300", "k_lens": "4096,2049,1000,100", "capacity": 0, "causal": True},
        # one long prompt: bound by the tensor cores and the exponentials
        {"name": "attention_long", "op": "attention", "heads": 16, "kv_heads": 4, "head_dim": 128, "dtype": "bf16",
         "q_lens": "16384", "k_lens": "16384", "capacity": 0, "causal": True},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["quantize", "linear", "attention", "attention"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "quantize":
        k = 32 * log(1, 256)
        return {"op": op, "rows": log(1, max(2, min(60000, 76_000_000 // k))), "k": k, "dtype": dtype}
    if op == "linear":
        n, k = 8 * log(16, 1376), 32 * log(2, 256)
        m = log(1, min(12480, 12480 * 11008 * 4096 // (n * k)))
        return {"op": op, "m": m, "n": n, "k": k, "bias": rng.random() < 0.5, "dtype": dtype}
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 1, 2, 3, 4, 5, 8])
    kind = rng.choice(["decode", "prompts", "chunks"])
    case = {"op": op, "heads": heads, "kv_heads": kv, "head_dim": rng.choice([64, 128]), "dtype": dtype}
    if dtype == "f32":  # the exact path: short sequences
        kind, longest = "prompts", 512
    elif kind == "decode":
        longest = log(16, 16384)
    else:
        longest = log(16, 8192)
    most = 1 if kind == "decode" else longest
    seqs = min(log(1, 48), max(1, 16 * 16384 * 16384 // (4 * heads * longest * most)), max(1, 300000 // longest))
    k_lens = [rng.randint(0 if seqs > 1 else 1, longest) for _ in range(seqs)]
    k_lens[rng.randrange(seqs)] = longest
    if kind == "decode":
        q_lens = [1] * seqs
    elif kind == "prompts":
        q_lens = list(k_lens)
    else:
        q_lens = [rng.randint(0, x) if rng.random() < 0.9 else min(longest, x + rng.randint(1, 9)) for x in k_lens]
        if not any(q_lens):
            q_lens[0] = 1
    return {**case, "q_lens": ",".join(map(str, q_lens)), "k_lens": ",".join(map(str, k_lens)),
            "capacity": longest if kind == "decode" else 0, "causal": rng.random() < 0.8}


def lengths(case):
    return [int(x) for x in case["q_lens"].split(",")], [int(x) for x in case["k_lens"].split(",")]


def work(case):
    if case["op"] == "quantize":
        n = case["rows"] * case["k"]
        # the rows, their codes and scales, and the values given back (bf16)
        return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + n // 2 + n // BLOCK + 2 * n, "flops": 4 * n}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * m * k + n * k // 2 + n * k // BLOCK + size * m * n + (4 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    size = 4 if case["dtype"] == "f32" else 2
    d, heads, kv = case["head_dim"], case["heads"], case["kv_heads"]
    q_lens, k_lens = lengths(case)
    seen = 0  # (query, key) pairs that the mask leaves
    for ql, kl in zip(q_lens, k_lens):
        if case["causal"]:
            first = max(0, ql - kl)  # queries before this one see nothing
            seen += sum((kl - ql + first + 1, kl)) * (ql - first) // 2 if ql > first else 0
        else:
            seen += ql * kl
    read = sum(kl for ql, kl in zip(q_lens, k_lens) if ql)
    return {"bytes": size * d * (2 * heads * sum(q_lens) + 2 * kv * read) + 4 * heads * sum(q_lens),
            "flops": 4 * d * heads * seen}


# ------------------------------------------------------------------------------ the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def hidden(rows, k):
        """Activations: unit normal, a few channels much larger (as behind a layer norm's scale)."""
        big = torch.where(torch.rand(k, generator=g, device="cuda") < 0.01, 16.0, 1.0)
        return normal(rows, k) * big

    st = {"case": case}
    if case["op"] == "quantize":
        rows, k = case["rows"], case["k"]
        st["x"] = hidden(rows, k).to(DTYPES[case["dtype"]])
        st["codes"] = torch.empty(rows, k // 2, dtype=torch.uint8, device="cuda")
        st["scales"] = torch.empty(scale_bytes(rows, k), dtype=torch.uint8, device="cuda")
        st["out"] = torch.empty(rows, k, dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        st["a"] = hidden(m, k).to(torch.bfloat16)
        # the weight as a program keeps it: codes, and the scales in their tiles
        st["w_codes"] = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
        exps = torch.randint(112, 119, (n, k // BLOCK), generator=g, device="cuda", dtype=torch.uint8)
        st["w_scales"] = tile_scales(exps)
        st["bias"] = normal(n) if case["bias"] else None
        st["codes"] = torch.empty(m, k // 2, dtype=torch.uint8, device="cuda")
        st["scales"] = torch.empty(scale_bytes(m, k), dtype=torch.uint8, device="cuda")
        st["out"] = torch.empty(m, n, dtype=DTYPES[case["dtype"]], device="cuda")
    else:
        q_lens, k_lens = lengths(case)
        heads, kv, d, cap = case["heads"], case["kv_heads"], case["head_dim"], case["capacity"]
        dt = DTYPES[case["dtype"]]
        nq = sum(q_lens)
        st["q_lens"], st["k_lens"] = q_lens, k_lens
        st["k_starts"] = [cap * i if cap else sum(k_lens[:i]) for i in range(len(k_lens))]
        nk = cap * len(k_lens) if cap else sum(k_lens)
        st["q"] = normal(nq, heads, d).to(dt)
        st["k"] = normal(max(nk, 1), kv, d).to(dt)
        st["v"] = normal(max(nk, 1), kv, d).to(dt)
        st["out"] = torch.empty(nq, heads, d, dtype=dt, device="cuda")
        st["lse"] = torch.empty(nq, heads, device="cuda")
        st["index"] = torch.tensor([q_lens, k_lens, st["k_starts"]], device="cuda")
    return st


# ------------------------------------------------------------------------------ layouts of the 4-bit data

def scale_bytes(rows, k):
    return -(-rows // 128) * -(-k // 128) * 512


def tile_scales(exps):
    """[rows][k / 32] scale bytes -> tiles of 128 rows x 4 blocks (512 bytes: row r of a tile at
    (r % 32) * 16 + (r // 32) * 4), padded with 0."""
    rows, nb = exps.shape
    p = torch.zeros(-(-rows // 128) * 128, -(-nb // 4) * 4, dtype=torch.uint8, device=exps.device)
    p[:rows, :nb] = exps
    return p.view(-1, 4, 32, p.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def untile_scales(tiles, rows, nb):
    t = tiles.view(-(-rows // 128), -(-nb // 4), 32, 4, 4).permute(0, 3, 2, 1, 4)
    return t.reshape(-(-rows // 128) * 128, -1)[:rows, :nb]


# ------------------------------------------------------------------------------ the plain forms

def power_of_two(e):
    """2^e in fp32 for whole e in [-127, 127]."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def plain_values(x):
    """The values that the 4-bit form of x's rows stands for, in fp32."""
    b = x.float().unflatten(1, (-1, BLOCK))
    e = (torch.frexp(b.abs().amax(2, keepdim=True))[1] - 3).clamp(-127, 127)
    a = b * power_of_two(-e)
    mag = a.abs().clamp(max=6.0)
    step = torch.where(mag < 2.0, 0.5, torch.where(mag < 4.0, 1.0, 2.0))
    return (torch.copysign(torch.round(mag / step) * step, a) * power_of_two(e)).flatten(1)


def plain_weight(codes, tiles):
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), 2).flatten(1)
    e = untile_scales(tiles, codes.shape[0], codes.shape[1] * 2 // BLOCK).to(torch.int32) - 127
    return (table[both.int()].unflatten(1, (-1, BLOCK)) * power_of_two(e).unsqueeze(2)).flatten(1)


def plain_attention(st):
    case = st["case"]
    kv, d = case["kv_heads"], case["head_dim"]
    group = case["heads"] // kv
    ql, kl, k_start = st["index"]
    q_start = ql.cumsum(0) - ql
    most_q, most_k, seqs = max(st["q_lens"]), max(max(st["k_lens"]), 1), len(st["q_lens"])
    t, j = torch.arange(most_q, device="cuda"), torch.arange(most_k, device="cuda")
    q = st["q"][(q_start[:, None] + t).clamp(max=st["q"].shape[0] - 1)].float()
    at = (k_start[:, None] + j).clamp(max=st["k"].shape[0] - 1)
    k, v = st["k"][at].float(), st["v"][at].float()
    q = q.view(seqs, most_q, kv, group, d).permute(0, 2, 3, 1, 4).reshape(seqs, kv, group * most_q, d)
    s = torch.matmul(q * d ** -0.5, k.permute(0, 2, 3, 1)).view(seqs, kv, group, most_q, most_k)
    last = kl[:, None] - ql[:, None] + t if case["causal"] else (kl[:, None] - 1).expand(seqs, most_q)
    seen = (j <= last[:, :, None]) & (j < kl[:, None, None])
    s.masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(4, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = s.sub_(top).exp_()
    total = p.sum(4, keepdim=True)
    o = torch.matmul(p.view(seqs, kv, group * most_q, most_k), v.permute(0, 2, 1, 3))
    o = o.view(seqs, kv, group, most_q, d) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(4)
    rows = st["q"].shape[0]
    seq = torch.repeat_interleave(torch.arange(seqs, device="cuda"), ql, output_size=rows)
    row = torch.arange(rows, device="cuda") - q_start[seq]
    out = o.permute(0, 3, 1, 2, 4)[seq, row].flatten(1, 2).to(st["q"].dtype)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2)[seq, row].flatten(1)}


def run(st):
    case = st["case"]
    if own:
        import long_video_diffusion_b200 as dp
        if case["op"] == "quantize":
            dp.mx4_quantize(st["x"], st["codes"], st["scales"])
            dp.mx4_dequantize(st["codes"], st["scales"], st["out"])
            return st["out"]
        if case["op"] == "linear":
            dp.mx4_quantize(st["a"], st["codes"], st["scales"])
            dp.mx4_linear(st["codes"], st["scales"], st["w_codes"], st["w_scales"], st["bias"], st["out"])
            return st["out"]
        dp.packed_attention(st["q"], st["k"], st["v"], st["q_lens"], st["k_lens"], st["out"], k_starts=st["k_starts"],
                            causal=case["causal"], lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    if case["op"] == "quantize":
        return plain_values(st["x"]).to(torch.bfloat16)
    if case["op"] == "linear":
        y = torch.matmul(plain_values(st["a"]), plain_weight(st["w_codes"], st["w_scales"]).T)
        if st["bias"] is not None:
            y += st["bias"]
        return y.to(st["out"].dtype)
    return plain_attention(st)


# ------------------------------------------------------------------------------ in 64 bits

def exact_values(x):
    out = []
    for part in x.split(max(1, (1 << 24) // x.shape[1])):
        b = part.double().reshape(part.shape[0], -1, BLOCK)
        # 2^-125 .. 2^127, exact: the last one that the largest magnitude reaches, a quarter of it
        powers = torch.tensor([2.0 ** e for e in range(-125, 128)], dtype=torch.float64, device=x.device)
        top = b.abs().max(dim=2, keepdim=True).values
        scale = powers[(torch.bucketize(top, powers, right=True) - 1).clamp(min=0)] / 4
        a = (b / scale).abs()
        code = ((a > 0.25).long() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
        grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
        out.append((grid[code] * torch.sign(b) * scale).reshape(part.shape))
    return torch.cat(out)


def exact_weight(st):
    codes, k = st["w_codes"], st["case"]["k"]
    n = codes.shape[0]
    w = torch.empty(n, k, dtype=torch.float64, device="cuda")
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    for half in (0, 1):
        c = (codes >> (4 * half)).long() & 15
        w[:, half::2] = torch.where(c >= 8, -grid[c % 8], grid[c % 8])
    r, b = torch.arange(n, device="cuda")[:, None], torch.arange(k // BLOCK, device="cuda")[None]
    at = ((r // 128) * -(-k // 128) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
    powers = torch.tensor([2.0 ** (e - 127) for e in range(255)], dtype=torch.float64, device="cuda")
    return w * powers[st["w_scales"][at].long()].repeat_interleave(BLOCK, 1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quantize":
        return exact_values(st["x"])
    if case["op"] == "linear":
        y = exact_values(st["a"]) @ exact_weight(st).T
        return y if st["bias"] is None else y + st["bias"].double()
    heads, d = case["heads"], case["head_dim"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for ql, kl, ks in zip(st["q_lens"], st["k_lens"], st["k_starts"]):
        blind = max(0, ql - kl) if case["causal"] else 0  # queries that see no key
        if kl and ql > blind:
            for h in range(heads):
                q = st["q"][at + blind:at + ql, h].double()
                k = st["k"][ks:ks + kl, h * case["kv_heads"] // heads].double()
                v = st["v"][ks:ks + kl, h * case["kv_heads"] // heads].double()
                s = q @ k.T / math.sqrt(d)
                if case["causal"]:
                    s = s + torch.full_like(s, -math.inf).triu(kl - (ql - blind) + 1)
                lse[at + blind:at + ql, h] = torch.logsumexp(s, 1)
                out[at + blind:at + ql, h] = torch.softmax(s, 1) @ v
        at += ql
    return {"out": out, "lse": lse}
