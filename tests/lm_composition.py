"""The recurrent core with attention, written out by hand in float64: forward,
and the backward formula by formula, with every value that the library hands on
in bfloat16 passed through `r`.  With r the identity it is the exact
composition (checked against autograd); with r = bf16 it is one sample of the
library's rounding noise, from which the tests take their bounds.  `broken`
leaves a part out or changes it, to show that the bounds see it.
"""
import math

import torch


def bf16(t):
    return t.to(torch.bfloat16).double()


def exact(t):
    return t


class Attention:
    def __init__(self, heads, kv_heads, hd, lens, window=0, freqs=None, mscale=1.0, pos=None):
        self.heads, self.kv_heads, self.hd, self.lens, self.window = heads, kv_heads, hd, list(lens), window
        self.freqs, self.mscale, self.pos = freqs, mscale, pos

    def turn(self, x, back):
        """Rows of heads turned by their positions (back: the other way)."""
        if self.freqs is None:
            return x
        ang = self.pos.double()[:, None] * self.freqs[None] * (2 * math.pi) * (-1 if back else 1)
        c, s = self.mscale * ang.cos()[:, None], self.mscale * ang.sin()[:, None]
        n = self.freqs.numel()
        y = x.reshape(x.shape[0], -1, self.hd)
        a, b = y[..., :n], y[..., n:2 * n]
        return torch.cat([a * c - b * s, a * s + b * c, y[..., 2 * n:]], -1).reshape(x.shape)

    def columns(self, qkv):
        q, k = self.heads * self.hd, (self.heads + self.kv_heads) * self.hd
        return qkv[:, :q], qkv[:, q:k], qkv[:, k:]

    def pairs(self):
        """(rows, columns of a query head, columns of its key head) of every softmax."""
        at = 0
        for n in self.lens:
            for h in range(self.heads):
                kh = h // (self.heads // self.kv_heads)
                yield (slice(at, at + n), slice(h * self.hd, (h + 1) * self.hd),
                       slice(kh * self.hd, (kh + 1) * self.hd))
            at += n

    def probabilities(self, q, k, broken):
        n = q.shape[0]
        s = q @ k.T / self.hd ** 0.5
        if broken == "flat scores":
            s = torch.zeros_like(s)
        keep = torch.ones(n, n, dtype=torch.bool).tril()
        if self.window and broken != "no window":
            keep = keep.triu(1 - self.window)
        return torch.softmax(s.masked_fill(~keep, -math.inf), -1)

    def forward(self, qkv, r, broken=None):
        """(rotated queries, keys), output; rows behind the last sequence get zeros."""
        q, k, v = self.columns(qkv)
        if broken != "no rotation":
            q, k = r(self.turn(q, False)), r(self.turn(k, False))
        out = torch.zeros_like(q)
        for rows, c, ck in self.pairs():
            out[rows, c] = r(self.probabilities(q[rows, c], k[rows, ck], broken)) @ v[rows, ck]
        return (q, k), r(out)

    def backward(self, datt, qk, v, out, r, broken=None):
        """Gradient of the unrotated Q|K|V rows."""
        q, k = qk
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        for rows, c, ck in self.pairs():
            p = self.probabilities(q[rows, c], k[rows, ck], broken)
            d = datt[rows, c]
            delta = (d * out[rows, c]).sum(1, keepdim=True)
            if broken == "no delta":
                delta = torch.zeros_like(delta)
            ds = r(p * (d @ v[rows, ck].T - delta))
            dq[rows, c] = ds @ k[rows, ck] / self.hd ** 0.5
            dk[rows, ck] += ds.T @ q[rows, c] / self.hd ** 0.5
            dv[rows, ck] += r(p).T @ d
        if broken == "dQ by 0.8":
            dq = 0.8 * dq
        if broken == "dK by 0.8":
            dk = 0.8 * dk
        if broken == "one head of a group in dV":
            dv = dv / (self.heads // self.kv_heads)
        dq, dk, dv = r(dq), r(dk), r(dv)
        if broken not in ("no inverse rotation", "no rotation"):
            dq, dk = r(self.turn(dq, broken != "rotated forward twice")), r(self.turn(dk, broken != "rotated forward twice"))
        return torch.cat([dq, dk, dv], 1)


BROKEN = ("flat scores", "no window", "no rotation", "no inverse rotation", "rotated forward twice", "no delta",
          "dQ by 0.8", "dK by 0.8", "one head of a group in dV", "no Q and K in dX", "no attention in dX")


def run(att, ops, x, dY, R, r=exact, broken=None):
    """R applications and their backward.  Of every application `attended` (what attention
    adds to the state) and `sent` (the gradient that comes back through it), and the
    blocks of the weights' gradients summed over the applications."""
    Wqkv, Wo, Wfc, Wproj = ops
    saved, y, res = [], r(x), {}
    for n in range(R):
        qkv = r(y @ Wqkv.T)
        qk, out = att.forward(qkv, r, broken)
        x1 = r(y + out @ Wo.T)
        pre = r(x1 @ Wfc.T)
        h = r(torch.relu(pre) ** 2)
        saved.append((y, qkv, qk, out, x1, pre, h))
        res["attended %d" % n] = x1 - y
        y = r(x1 + h @ Wproj.T)
    res["out"] = y
    g = r(dY)
    dW = [torch.zeros_like(w) for w in ops]
    for n in reversed(range(R)):
        y0, qkv, qk, out, x1, pre, h = saved[n]
        dpre = r((g @ Wproj) * 2 * torch.relu(pre))
        dx1 = r(g + dpre @ Wfc)
        datt = r(dx1 @ Wo)
        dqkv = att.backward(datt, qk, att.columns(qkv)[2], out, r, broken)
        through = dqkv @ Wqkv
        if broken == "no Q and K in dX":
            first = dqkv.shape[1] - att.kv_heads * att.hd
            through = dqkv[:, first:] @ Wqkv[first:]
        if broken == "no attention in dX":
            through = torch.zeros_like(through)
        dx = r(dx1 + through)
        res["sent %d" % n] = dx - dx1
        for w, (a, b) in zip(dW, ((dqkv, y0), (dx1, out), (dpre, x1), (g, h))):
            w += a.T @ b
        g = dx
    res["dX"] = g
    q, k = att.heads * att.hd, (att.heads + att.kv_heads) * att.hd
    res.update(dWq=dW[0][:q], dWk=dW[0][q:k], dWv=dW[0][k:], dWo=dW[1], dWfc=dW[2], dWproj=dW[3])
    return res


def off(got, want):
    """Per result, the distance relative to the size of what it should be."""
    return {n: float((got[n] - want[n]).norm() / want[n].norm()) for n in want}
