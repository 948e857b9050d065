"""Seeded inputs for the calls under logit rules: logits with special values,
ragged token histories (empty, of one token, with repeats, with ids outside
the vocabulary), biases and grammars (rows that allow everything, one entry,
nothing)."""
import numpy as np

import synth

DTYPES = ("bf16", "fp16", "fp32")
EPS = {"bf16": 2.0 ** -7, "fp16": 2.0 ** -10, "fp32": 2.0 ** -23}  # torch.finfo(t).eps


def to_bits(x, dtype):
    x = x.astype(np.float32)
    return {"bf16": synth.f32_to_bf16_bits, "fp16": synth.f32_to_fp16_bits, "fp32": lambda a: a}[dtype](x)


class Rules:
    """One batch: arrays as the library takes them, lists as the oracle does."""

    def __init__(self, T, V, dtype, seed, L=60, shared=False, history=True, bias=True, grammar=True, empty_row=True,
                 extra_cols=0, extra_len=0):
        rng = np.random.default_rng(seed)
        self.T, self.V, self.dtype = T, V, dtype
        self.bits = to_bits(rng.normal(0, 3, (T, V + extra_cols)), dtype)
        self.targets = rng.integers(0, V, T).astype(np.int64)
        self.mask = (rng.random(T) < 0.8).astype(np.uint8)
        self.args, self.oracle = {}, {}
        if history:
            B = max(1, T // 3) if shared else T
            # few different ids, so that they repeat; some outside [0, V)
            pool = np.concatenate([rng.integers(0, V, 12), [0, V - 1, -1, V, 2**31 - 1, -2**31]])
            tok = rng.choice(pool, (B, L + extra_len)).astype(np.int32)
            hist = rng.integers(0, L + 1, T)
            hist[0] = L
            if T > 1:
                hist[1] = 0
            if T > 2:
                hist[2] = 1
            prompt = (hist * rng.random(T)).astype(np.int64)
            seq = rng.integers(0, B, T) if shared else np.arange(T)
            rho = rng.uniform(0.7, 1.6, T).astype(np.float32)
            f, p = (rng.uniform(-0.5, 1.0, T).astype(np.float32) for _ in range(2))
            self.tokens = tok
            self.args.update(hist_len=hist.astype(np.int32), prompt_len=prompt.astype(np.int32), repetition=rho,
                             frequency=f, presence=p)
            if shared:
                self.args["row_seq"] = seq.astype(np.int32)
            self.oracle.update(prompts=[tok[seq[t], :prompt[t]] for t in range(T)],
                               outputs=[tok[seq[t], prompt[t]:hist[t]] for t in range(T)],
                               repetition=rho, frequency=f, presence=p)
        if bias:
            n = rng.integers(0, 7, T)
            n[-1] = 0
            off = np.concatenate([[0], np.cumsum(n)]).astype(np.int64)
            ids = rng.integers(-1, V + 1, off[-1]).astype(np.int32)
            if off[1] > 1:
                ids[1] = ids[0]  # listed twice: the last one counts
            val = rng.normal(0, 2, off[-1]).astype(np.float32)
            self.args.update(bias_offsets=off, bias_tokens=ids, bias_values=val)
            self.oracle["biases"] = [list(zip(ids[off[t]:off[t + 1]], val[off[t]:off[t + 1]])) for t in range(T)]
        if grammar:
            ok = rng.random((T, V)) < rng.choice([0.1, 0.5, 0.95], (T, 1))
            ok[0] = True
            ok[np.arange(T), self.targets] = True
            if T > 3:
                ok[3] = False
                ok[3, self.targets[3]] = True
            if T > 4 and empty_row:
                ok[4] = False
            W = (V + 31) // 32
            full = np.ones((T, W * 32), dtype=bool)  # bits past V are set and must not matter
            full[:, :V] = ok
            words = (full.reshape(T, W, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(2)
            self.args["allowed"] = words.astype(np.uint32).view(np.int32)
            self.oracle["allowed"] = ok

    def logits64(self):
        from oracle import lp_oracle as O
        return O.widen(self.bits, self.dtype)[:, :self.V]

    def plant_specials(self, seed=5):
        """NaN and infinities where the grammar does not look, the type's lowest value and -inf where it does."""
        rng = np.random.default_rng(seed)
        low = {"bf16": 0xff7f, "fp16": 0xfbff, "fp32": np.float32(-3.4028234e38)}[self.dtype]
        odd = {"bf16": (0x7fc0, 0x7f80, 0xff80), "fp16": (0x7e00, 0x7c00, 0xfc00),
               "fp32": (np.float32(np.nan), np.float32(np.inf), np.float32(-np.inf))}[self.dtype]
        ok = self.oracle["allowed"]
        for t in range(self.T):
            shut = np.nonzero(~ok[t])[0]
            for j in shut[:3 * len(odd)]:
                self.bits[t, j] = odd[rng.integers(0, 3)]
            free = [j for j in np.nonzero(ok[t])[0] if j != self.targets[t]]
            for j in free[:4]:
                self.bits[t, j] = low if rng.random() < 0.5 else odd[2]
        return self

    def device(self):
        """(logits tensor [T, V] viewing the wider buffer, LogitRules) on the GPU."""
        import entropy_chunked_row_amd as lp
        from tests.helpers import to_dev, to_dev_bits
        x = to_dev(self.bits) if self.dtype == "fp32" else to_dev_bits(self.bits, self.dtype)
        kw = {k: to_dev(v) for k, v in self.args.items()}
        if hasattr(self, "tokens"):
            L = int(self.args["hist_len"].max()) if self.args["hist_len"].size else 0
            kw["tokens"] = to_dev(self.tokens)[:, :max(L, 1)]
        return x[:, :self.V], lp.LogitRules(**kw)

    def processed(self):
        from oracle import lp_oracle as O
        with np.errstate(invalid="ignore", over="ignore"):
            return O.apply_rules(self.logits64(), **self.oracle)
