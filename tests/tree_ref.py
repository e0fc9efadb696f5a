"""FP64 references of the speculative-decoding calls (tests only): attention of
tree nodes over an oracle cache, and sequential block tables and slot maps."""
import numpy as np

HEAD_DIM = 128


def cached_kv(ora, b, L):
    """K, V float64 [hkv][L][128] of sequence b's cached tokens."""
    cold = max(0, L - ora.hot)
    out = np.zeros((2, ora.hkv, L, HEAD_DIM))
    for i in range(-(-cold // ora.block)):
        if ora.quant_bits == 0:
            _, vals = ora.get_block_fp16(b, i)
            vals = vals.astype(np.float64)
        else:
            _, codes, sc = ora.get_block(b, i)
            vals = codes.astype(np.float64) * sc.astype(np.float64)[:, :, None, None]
        p0, n = i * ora.block, min(ora.block, cold - i * ora.block)
        out[:, :, p0:p0 + n] = vals.transpose(1, 0, 2, 3)[:, :, :n]
    ring = ora.ring(b).astype(np.float64)  # [hkv][hot][2][128]
    pos = np.arange(cold, L)
    out[:, :, cold:] = ring[:, pos % ora.hot].transpose(2, 0, 1, 3)
    return out[0], out[1]


def tree_attention(k, v, q, k_tree, v_tree, mask, n_tree, scale):
    """One sequence: k, v float64 [hkv][L][128] cached; q [nodes][hq][128],
    k_tree, v_tree [nodes][hkv][128], mask int64 [nodes].  Returns out
    [n_tree][hq][128], lse [n_tree][hq] and the bounds (tol_out, tol_lse) on
    the error of a kernel that rounds each softmax weight once to FP16, sums in
    FP32 and rounds the output once to FP16:
      dz    = 128 * 2^-24 * max_j sum_c |q_c k_jc| * |scale|: a logit's 128
              FP32 additions (a relative 2 dz of numerator and denominator);
      out   : half a step of the output, 2^-11 |o|, and of each weight, 2^-11
              sum_j p_j |v_j|; a weight below 2^-14 of the largest is subnormal
              and rounded by at most 2^-25 of it: N 2^-25 max|v|;
      lse   : dz, N 2^-24 for the sum of N weights, and the rounding of the
              result, 2^-21 max(1, |lse|)."""
    nodes, hq = q.shape[:2]
    g = hq // k.shape[0]
    L = k.shape[1]
    f = lambda x: np.asarray(x, np.float64)  # noqa: E731
    o = np.zeros((n_tree, hq, HEAD_DIM))
    lse = np.full((n_tree, hq), -np.inf)
    tol_o, tol_l = np.zeros_like(o), np.zeros_like(lse)
    m = np.asarray(mask).view(np.uint64)
    for t in range(n_tree):
        on = [j for j in range(n_tree) if (int(m[t]) >> j) & 1]
        for h in range(hq):
            kk = np.concatenate([k[h // g], f(k_tree)[on, h // g]])
            vv = np.concatenate([v[h // g], f(v_tree)[on, h // g]])
            if L + len(on) == 0:
                continue
            qq = f(q)[t, h]
            z = kk @ qq * scale
            top = z.max()
            p = np.exp(z - top)
            lse[t, h] = top + np.log(p.sum())
            p /= p.sum()
            o[t, h] = p @ vv
            n = len(z)
            dz = 128 * 2.0 ** -24 * (np.abs(kk) @ np.abs(qq)).max() * abs(scale)
            spread = p @ np.abs(vv)
            tol_o[t, h] = 2.0 ** -11 * np.abs(o[t, h]) + (2.0 ** -11 + 2 * dz) * spread \
                + n * 2.0 ** -25 * np.abs(vv).max() + 2.0 ** -25
            tol_l[t, h] = dz + n * 2.0 ** -24 + 2.0 ** -21 * max(1.0, abs(lse[t, h]))
    return o, lse, tol_o, tol_l


def random_masks(rng, batch, nodes, kind):
    """int64 masks [batch][nodes]: "tree" (ancestors of a random tree), "any"
    (any bits, rows without any among them) or "empty"."""
    from int8_paged_kv_hybrid_b200 import tree_masks
    if kind == "tree":
        parents = np.stack([[int(rng.integers(-1, t)) if t else -1 for t in range(nodes)] for _ in range(batch)])
        return tree_masks(parents)
    m = np.zeros((batch, nodes), np.uint64)
    if kind == "any":
        m = rng.integers(0, 2 ** 64, size=(batch, nodes), dtype=np.uint64)
        m[:, ::3] = 0
    return m.view(np.int64)


class PoolModel:
    """Block tables of hyb_pool_resize, one sequence after the other."""

    def __init__(self, batch, phys, width, hot, block):
        self.width, self.hot, self.block, self.phys = width, hot, block, phys
        self.free = list(range(phys))
        self.head = 0
        self.held = [[] for _ in range(batch)]

    def resize(self, lens):
        """Returns the sequences that were refused for want of blocks."""
        avail, refused, given = list(self.free), [], []
        asked = 0
        taken = 0
        for b, n in enumerate(lens):
            want = -(-max(0, n - self.hot) // self.block) if n >= 0 else len(self.held[b])
            if want > self.width:
                want = len(self.held[b])
            need = want - len(self.held[b])
            if need > 0:
                asked += need
                if asked > len(avail):
                    refused.append(b)
                    continue
                self.held[b] += avail[taken:taken + need]
                taken += need
            elif need < 0:
                given += self.held[b][want:]
                self.held[b] = self.held[b][:want]
        self.free = avail[taken:] + given
        self.head = (self.head + taken) % self.phys
        return refused


def slot_map(table, lens, first, n_tok, hot, block):
    cu, out = [0], []
    for b in range(len(lens)):
        for p in range(first[b], first[b] + max(0, n_tok[b])):
            if p < 0 or p >= lens[b]:
                out.append(-1)
            elif p >= lens[b] - hot:
                out.append(-2 - (b * hot + p % hot))
            else:
                out.append(int(table[b][p // block]) * block + p % block)
        cu.append(len(out))
    return np.array(cu, np.int32), np.array(out, np.int64)
