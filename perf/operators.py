"""Measured cases of the operators around the vocabulary.

Four operators, each in a plain form (elementary torch operations in fp32, in
fp64 where fp32 loses what matters) and, where `own` is true, through this
package's entry points:

* process  -- penalties for repeated tokens, sparse biases and a grammar mask on logits (a decode step);
* score    -- log-prob, entropy and log-sum-exp of the distribution those rules leave, and score_grad its
              gradient with respect to the raw logits (training on what was sampled from it);
* embed    -- embedding lookup with a scale, and embed_grad its weight gradient by sorted tokens (the other end of
              a tied output head);
* w4       -- logits of few rows through an output head held in 4 bits with group scales.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NEG_INF = float("-inf")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one request of a serving loop: a single row, a short history, a few biases, a grammar
        dict(name="process_one_row", kind="process", dtype="bf16", T=1, V=151936, S=1, L=517, prompt=211, bias=3,
             grammar=True),
        # a full decode batch with long ragged histories, one token buffer a request
        dict(name="process_batch", kind="process", dtype="fp16", T=256, V=129280, S=256, L=4096, prompt=1500, bias=40,
             grammar=True),
        # a handful of odd fp32 rows, no grammar
        dict(name="score_odd_rows", kind="score", dtype="fp32", T=5, V=20011, S=5, L=333, prompt=100, bias=2,
             grammar=False, tau=1.0),
        # scoring whole rollouts: 8 sequences of 1024 sampled tokens, every position sees its own prefix
        dict(name="score_rollouts", kind="score", dtype="bf16", T=8192, V=151936, S=8, L=1536, prompt=512, bias=24,
             grammar=True, tau=0.7),
        # the gradient of a small ragged batch
        dict(name="score_grad_small", kind="score_grad", dtype="fp16", T=37, V=4099, S=3, L=200, prompt=64, bias=4,
             grammar=True, tau=1.3),
        # the gradient of one training step's rollouts
        dict(name="score_grad_rollouts", kind="score_grad", dtype="bf16", T=4096, V=151936, S=4, L=1536, prompt=512,
             bias=24, grammar=True, tau=0.7),
        # the token embeddings of a packed training batch
        dict(name="embed_batch", kind="embed", dtype="bf16", N=32768, h=5120, V=151936),
        # the embedding gradient of a toy model
        dict(name="embed_grad_tiny", kind="embed_grad", dtype="fp32", N=64, h=256, V=1024),
        # the embedding gradient of a packed training batch: frequent tokens come up thousands of times
        dict(name="embed_grad_batch", kind="embed_grad", dtype="bf16", N=32768, h=5120, V=151936),
        # the head of a single decoded token
        dict(name="w4_one_row", kind="w4", dtype="bf16", out="bf16", T=1, h=5120, V=151936, group=128),
        # the head of a small decode batch
        dict(name="w4_few_rows", kind="w4", dtype="bf16", out="fp32", T=8, h=5120, V=151936, group=64),
        # the head of a ragged decode batch, small groups, fp32 logits
        dict(name="w4_batch", kind="w4", dtype="fp16", out="fp32", T=40, h=7168, V=129280, group=32),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["process", "score", "score_grad", "embed", "embed_grad", "w4", "w4"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    if kind in ("process", "score", "score_grad"):
        V = _spread(rng, 1000, 151936)
        most = {"process": 256, "score": 8192, "score_grad": 4096}[kind]
        T = _spread(rng, 1, most if dtype != "fp32" else most // 2)
        S = T if kind == "process" else rng.randint(1, min(T, 8))
        made = -(-T // S)
        prompt = rng.randint(0, 2048 if kind == "process" else 512)
        L = prompt + (rng.randint(1, 2048) if kind == "process" else made)
        return dict(kind=kind, dtype=dtype, T=T, V=V, S=S, L=L, prompt=prompt, bias=rng.randint(0, 40),
                    grammar=rng.random() < 0.7, tau=rng.choice([1.0, 0.7, rng.uniform(0.3, 2.0)]))
    if kind in ("embed", "embed_grad"):
        half = 1 if dtype != "fp32" else 2
        return dict(kind=kind, dtype=dtype, N=_spread(rng, 1, 32768 // half), h=_spread(rng, 64, 5120 // half),
                    V=_spread(rng, 100, 151936))
    return dict(kind=kind, dtype=rng.choice(["bf16", "fp16"]), out=rng.choice(["bf16", "fp16", "fp32"]),
                T=_spread(rng, 1, 40), h=32 * _spread(rng, 2, 160), V=_spread(rng, 100, 129280),
                group=rng.choice([32, 64, 128]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _tokens(shape, V, gen):
    """Token ids with the skew of text: a few ids make up most of it."""
    u = torch.rand(shape, generator=gen, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(V)).long().clamp_(1, V) - 1
    return (rank * 7919 + 13) % V if V % 7919 else rank


def _rules(c, gen):
    T, V, S, L = c["T"], c["V"], c["S"], c["L"]
    s = {"tokens": _tokens((S, max(L, 1)), V, gen).int()}
    row = torch.arange(T, device="cuda")
    made = -(-T // S)
    if c["kind"] == "process":
        # ragged requests: every row its own buffer, prompt and length
        s["row_seq"] = None
        s["prompt_len"] = torch.randint(0, c["prompt"] + 1, (T,), generator=gen, device="cuda").int()
        more = torch.rand(T, generator=gen, device="cuda") * (L - s["prompt_len"] + 1)
        s["hist_len"] = (s["prompt_len"] + more.int()).clamp_(max=L)
    else:
        # rollouts: row t is position t % made of sequence t // made and sees that sequence's prefix
        s["row_seq"] = (row // made).int()
        s["prompt_len"] = torch.full((T,), c["prompt"], dtype=torch.int32, device="cuda")
        s["hist_len"] = (c["prompt"] + row % made).int()
    rand = lambda: torch.rand(T, generator=gen, device="cuda")  # noqa: E731
    s["repetition"] = 1.0 + 0.3 * rand()
    s["frequency"] = 0.5 * rand()
    s["presence"] = 0.5 * rand()
    s["bias_offsets"] = s["bias_tokens"] = s["bias_values"] = None
    if c["bias"]:
        # `bias` different ids a row, from a start of the row's own
        nb = min(c["bias"], V)
        start = torch.randint(0, V, (T, 1), generator=gen, device="cuda")
        ids = (start + torch.arange(nb, device="cuda") * max(1, V // nb)) % V
        s["bias_offsets"] = torch.arange(T + 1, device="cuda") * nb
        s["bias_tokens"] = ids.reshape(-1).int()
        s["bias_values"] = torch.randn(T * nb, generator=gen, device="cuda") * 2.0
    s["targets"] = torch.randint(0, V, (T,), generator=gen, device="cuda")
    s["allowed"] = None
    if c["grammar"]:
        # three tokens of four allowed, one row of eight down to one of four; what was sampled is allowed
        W = (V + 31) // 32
        word = lambda: torch.randint(-2**31, 2**31, (T, W), generator=gen, device="cuda").int()  # noqa: E731
        a, b = word(), word()
        bits = torch.where((row % 8 == 7)[:, None], a & b, a | b)
        w = s["targets"] // 32
        one = (1 << (s["targets"] % 32)).to(torch.int64)
        old = bits.gather(1, w[:, None]).long() & 0xffffffff
        new = old | one[:, None]
        new = torch.where(new >= 2**31, new - 2**32, new)
        s["allowed"] = bits.scatter_(1, w[:, None], new.int())
    return s


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)
    kind = c["kind"]
    dt = DTYPES[c["dtype"]]
    randn = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    s = {"case": c}
    if kind in ("process", "score", "score_grad"):
        s["logits"] = (randn(c["T"], c["V"]) * 3.0).to(dt)
        s.update(_rules(c, gen))
        if kind == "score_grad":
            # what the forward left: log-sum-exp and entropy, fp32
            _, s["entropy"], s["lse"] = _plain_score(s, c["tau"])
            s["grad_logprob"] = randn(c["T"])
            s["grad_entropy"] = 0.1 * randn(c["T"])
        return s
    if kind in ("embed", "embed_grad"):
        s["tokens"] = _tokens((c["N"],), c["V"], gen)
        s["scale"] = math.sqrt(c["h"])
        if kind == "embed":
            s["weight"] = (randn(c["V"], c["h"]) * 0.02).to(dt)
        else:
            s["grad_out"] = (randn(c["N"], c["h"]) * 0.01).to(dt)
        return s
    s["hidden"] = randn(c["T"], c["h"]).to(dt)
    # two 4-bit values a byte, the even column in the low half, each its whole number -8 .. 7 plus 8
    s["packed"] = torch.empty(c["V"], c["h"] // 2, dtype=torch.uint8, device="cuda")
    part = max(1, (1 << 27) // c["h"])
    for v in range(0, c["V"], part):
        q = (randn(min(part, c["V"] - v), c["h"]) * 2.3).round_().clamp_(-8, 7).add_(8).to(torch.uint8)
        s["packed"][v:v + part] = q[:, 0::2] | (q[:, 1::2] << 4)
    groups = -(-c["h"] // c["group"])
    s["scales"] = (0.008 * (0.5 + torch.rand(c["V"], groups, generator=gen, device="cuda"))).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _counts(s, T, V):
    """(seen in prompt or output [T, V], times in the output [T, V] fp32) of every row's history."""
    tok = s["tokens"].long()
    if s["row_seq"] is not None:
        tok = tok[s["row_seq"].long()]
    at = torch.arange(tok.shape[1], device=tok.device)
    live = (at < s["hist_len"][:, None]) & (tok >= 0) & (tok < V)
    made = live & (at >= s["prompt_len"][:, None])
    one = torch.ones((), device=tok.device).expand(tok.shape)
    times = torch.zeros(T, V + 1, device=tok.device).scatter_add_(1, torch.where(made, tok, V), one)[:, :V]
    seen = torch.zeros(T, V + 1, device=tok.device).scatter_(1, torch.where(live, tok, V), 1.0)[:, :V] > 0
    return seen, times


def _bias(s, T, V):
    n = s["bias_tokens"].numel()
    row = torch.repeat_interleave(torch.arange(T, device="cuda"), s["bias_offsets"].diff(), output_size=n)
    b = torch.zeros(T, V, device="cuda")
    b[row, s["bias_tokens"].long()] = s["bias_values"]
    return b


def _allowed(s, V):
    bit = torch.arange(32, device="cuda", dtype=torch.int32)
    return ((s["allowed"][:, :, None] >> bit) & 1).bool().flatten(1)[:, :V]


def _plain_processed(s):
    z = s["logits"].float()
    T, V = z.shape
    seen, times = _counts(s, T, V)
    rep = s["repetition"][:, None]
    z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
    z = z - s["frequency"][:, None] * times
    z = z - s["presence"][:, None] * (times > 0)
    if s["bias_tokens"] is not None:
        z = z + _bias(s, T, V)
    if s["allowed"] is not None:
        z = z.masked_fill(~_allowed(s, V), NEG_INF)
    return z


def _plain_score(s, tau):
    z = _plain_processed(s) / tau
    m = z.amax(1, keepdim=True)
    lse = (m + (z - m).exp().sum(1, keepdim=True).log())[:, 0]
    logp = z - lse[:, None]
    H = -(logp.exp() * logp.masked_fill(logp == NEG_INF, 0.0)).sum(1)
    return logp.gather(1, s["targets"][:, None])[:, 0], H, lse


def _plain_score_grad(s, tau):
    z = _plain_processed(s) / tau
    logp = z - s["lse"][:, None]
    p = logp.exp()
    g = s["grad_logprob"][:, None]
    d = -g * p
    d.scatter_add_(1, s["targets"][:, None], g)
    logp = logp.masked_fill_(logp == NEG_INF, 0.0)
    d -= s["grad_entropy"][:, None] * p * (logp + s["entropy"][:, None])
    d /= tau
    seen, _ = _counts(s, *z.shape)
    rep = s["repetition"][:, None]
    d = torch.where(seen, torch.where(s["logits"] > 0, d / rep, d * rep), d)
    if s["allowed"] is not None:
        d = d.masked_fill(~_allowed(s, z.shape[1]), 0.0)
    return d.to(s["logits"].dtype)


def _plain_w4(s, c):
    q = s["packed"]
    w = torch.stack((q & 15, q >> 4), 2).flatten(1).float() - 8.0
    w = w * s["scales"].float().repeat_interleave(c["group"], 1)[:, :c["h"]]
    return (s["hidden"].float() @ w.t()).to(DTYPES[c["out"]])


def _plain(s):
    c, kind = s["case"], s["case"]["kind"]
    if kind == "process":
        return _plain_processed(s).to(s["logits"].dtype)
    if kind == "score":
        return _plain_score(s, c["tau"])
    if kind == "score_grad":
        return _plain_score_grad(s, c["tau"])
    if kind == "embed":
        return (s["weight"][s["tokens"]].float() * s["scale"]).to(s["weight"].dtype)
    if kind == "embed_grad":
        g = torch.zeros(c["V"], c["h"], device="cuda")
        return g.index_add_(0, s["tokens"], s["grad_out"].float() * s["scale"])
    return _plain_w4(s, c)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _own(s):
    import entropy_chunked_row_amd as lp

    c, kind = s["case"], s["case"]["kind"]
    if kind in ("process", "score", "score_grad"):
        rules = lp.LogitRules(tokens=s["tokens"], hist_len=s["hist_len"], prompt_len=s["prompt_len"],
                              row_seq=s["row_seq"], repetition=s["repetition"], frequency=s["frequency"],
                              presence=s["presence"], bias_offsets=s["bias_offsets"], bias_tokens=s["bias_tokens"],
                              bias_values=s["bias_values"], allowed=s["allowed"])
        if kind == "process":
            return lp.lp_process_logits(s["logits"], rules)
        if kind == "score":
            return lp.lp_processed_logprobs_entropy(s["logits"], rules, s["targets"], None, c["tau"])
        return lp.lp_processed_logprobs_entropy_backward(s["logits"], rules, s["targets"], None, c["tau"], s["lse"],
                                                         s["entropy"], s["grad_logprob"], s["grad_entropy"])
    if kind == "embed":
        return lp.lp_embedding(s["weight"], s["tokens"], s["scale"])
    if kind == "embed_grad":
        return lp.lp_embedding_backward(s["grad_out"], s["tokens"], c["V"], s["scale"])
    return lp.lp_lm_head_w4_logits(s["hidden"], s["packed"], s["scales"], c["group"], out_dtype=DTYPES[c["out"]])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c, kind = case, case["kind"]
    size = 4 if c["dtype"] == "fp32" else 2
    if kind in ("process", "score", "score_grad"):
        T, V = c["T"], c["V"]
        n = T * V
        rules = 4 * c["S"] * c["L"] + 8 * T * c["bias"] + 24 * T + (n // 8 if c["grammar"] else 0)
        if kind == "process":
            return {"bytes": 2 * n * size + rules, "flops": 3 * n}
        if kind == "score":
            return {"bytes": n * size + rules + 20 * T, "flops": 6 * n}
        return {"bytes": 2 * n * size + rules + 24 * T, "flops": 9 * n}
    if kind == "embed":
        return {"bytes": 2 * c["N"] * c["h"] * size + 8 * c["N"], "flops": c["N"] * c["h"]}
    if kind == "embed_grad":
        return {"bytes": c["N"] * c["h"] * size + 8 * c["N"] + 4 * c["V"] * c["h"], "flops": 2 * c["N"] * c["h"]}
    head = c["V"] * c["h"] // 2 + 2 * c["V"] * -(-c["h"] // c["group"])
    out = 4 if c["out"] == "fp32" else 2
    return {"bytes": head + c["T"] * (c["h"] * size + c["V"] * out), "flops": 2 * c["T"] * c["h"] * c["V"]}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_rows(s, r):
    """(processed logits fp64, d processed / d raw) of row r."""
    z = s["logits"][r].double()
    V = z.numel()
    buf = s["tokens"][r if s["row_seq"] is None else int(s["row_seq"][r])].long()
    n, n0 = int(s["hist_len"][r]), int(s["prompt_len"][r])
    rep, f, p = (s[k][r].double() for k in ("repetition", "frequency", "presence"))
    times = torch.bincount(buf[n0:n], minlength=V).double()
    seen = torch.bincount(buf[:n], minlength=V) > 0
    slope = torch.ones_like(z)
    slope[seen] = torch.where(z[seen] > 0, 1.0 / rep, rep)
    z = z * slope - f * times - p * times.clamp(max=1.0)
    if s["bias_tokens"] is not None:
        a, b = int(s["bias_offsets"][r]), int(s["bias_offsets"][r + 1])
        z[s["bias_tokens"][a:b].long()] += s["bias_values"][a:b].double()
    if s["allowed"] is not None:
        j = torch.arange(V, device="cuda")
        shut = torch.bitwise_right_shift(s["allowed"][r][j // 32].long(), j % 32) % 2 == 0
        z[shut] = NEG_INF
        slope[shut] = 0.0
    return z, slope


def exact(case, seed):
    c, kind = case, case["kind"]
    s = prepare(case, seed)
    if kind in ("process", "score", "score_grad"):
        if c["T"] > 8192 or (kind != "score" and c["T"] * c["V"] > 1 << 30):
            return None
        rows = []
        for r in range(c["T"]):
            z, slope = _exact_rows(s, r)
            if kind == "process":
                rows.append(z)
                continue
            z = z / c["tau"]
            if kind == "score":
                lse = torch.logsumexp(z, 0)
                logp = z - lse
                e = torch.special.entr(logp.exp()).sum()
                rows.append(torch.stack((logp[s["targets"][r]], e, lse)))
                continue
            logp = z - s["lse"][r].double()
            p = logp.exp()
            g, gh = s["grad_logprob"][r].double(), s["grad_entropy"][r].double()
            d = gh * (torch.special.entr(p) - p * s["entropy"][r].double()) - g * p
            d[s["targets"][r]] += g
            rows.append(d * slope / c["tau"])
        got = torch.stack(rows)
        return tuple(got.t().contiguous()) if kind == "score" else got
    if kind == "embed":
        return torch.nn.functional.embedding(s["tokens"], s["weight"]).double() * s["scale"]
    if kind == "embed_grad":
        ids, back = s["tokens"].unique(return_inverse=True)
        g = torch.zeros(ids.numel(), c["h"], dtype=torch.float64, device="cuda")
        g.index_add_(0, back, s["grad_out"].double())
        out = torch.zeros(c["V"], c["h"], dtype=torch.float64, device="cuda")
        out[ids] = g * s["scale"]
        return out
    x = s["hidden"].double()
    out = torch.zeros(c["T"], c["V"], dtype=torch.float64, device="cuda")
    for k in range(0, c["h"], c["group"]):
        e = min(k + c["group"], c["h"])
        q = s["packed"][:, k // 2:e // 2].long()
        dot = (x[:, k:e:2] @ (q % 16 - 8).double().t()) + (x[:, k + 1:e:2] @ (q // 16 - 8).double().t())
        out += dot * s["scales"][:, k // c["group"]].double()
    return out
