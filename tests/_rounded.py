"""Arrays in 64 bits beside a bound on what an f32 evaluation of the same steps may be off by: every operation
rounds once (half a unit, 2^-24 relative), a sum of n terms in any order n times.  Fused and fewer roundings stay
within the bound."""
import numpy as np

U = 2.0 ** -24


class A:
    def __init__(self, v, e=0.0):
        self.v = np.asarray(v, np.float64)
        self.e = np.broadcast_to(np.asarray(e, np.float64), self.v.shape)

    @staticmethod
    def of(x):
        return x if isinstance(x, A) else A(x)

    def __add__(self, o):
        o = A.of(o)
        v, e = self.v + o.v, self.e + o.e
        return A(v, e + U * (np.abs(v) + e))

    def __neg__(self):
        return A(-self.v, self.e)

    def __sub__(self, o):
        return self + (-A.of(o))

    def __mul__(self, o):
        o = A.of(o)
        v = self.v * o.v
        e = np.abs(self.v) * o.e + np.abs(o.v) * self.e + self.e * o.e
        return A(v, e + U * (np.abs(v) + e))

    def sum(self, axis, keepdims=False):
        n = self.v.shape[axis]
        e, s = self.e.sum(axis, keepdims=keepdims), np.abs(self.v).sum(axis, keepdims=keepdims)
        return A(self.v.sum(axis, keepdims=keepdims), e + n * U * (s + e))

    def mean(self):
        return self.sum(1, True) * (1.0 / self.v.shape[1])

    def rsqrt(self, least):
        """least: what the argument cannot be below whatever the errors (a sum of squares is not negative).  The
        function falls: an argument within [lo, v + e] gives a value between theirs."""
        lo = np.maximum(self.v - self.e, least * (1 - 2 * U))
        v = self.v ** -0.5
        e = np.maximum(lo ** -0.5 - v, v - (self.v + self.e) ** -0.5)
        return A(v, e + 4 * U * (v + e))


NONE, RMS, LAYER = range(3)


def hat(v, kind, eps):
    """(normalised rows, their factor)."""
    if kind == LAYER:
        v = v - v.mean()
    r = ((v * v).mean() + eps).rsqrt(eps)
    return v * r, r


def norm(v, kind, w, b, eps):
    if kind == NONE:
        return v
    v = hat(v, kind, eps)[0]
    if w is not None:
        v = v * w
    return v if b is None else v + b


def forward(x, y, res, gate, post, wp, bp, pre, wn, bn, eps):
    """(Z, N or None)"""
    z = A.of(x) * res
    if y is not None:
        u = norm(A.of(y), post, wp, bp, eps)
        z = z + (u if gate is None else u * gate)
    return z, norm(z, pre, wn, bn, eps) if pre != NONE else None


def _back(v, d, kind, w, eps):
    """(gradient of v, terms of the weight's, terms of the bias's)"""
    if kind == NONE:
        return d, None, None
    h, r = hat(v, kind, eps)
    dh = d if w is None else d * w
    dv = dh - h * (dh * h).mean()
    if kind == LAYER:
        dv = dv - dh.mean()
    return dv * r, d * h, d


def backward(z, dz, dn, y, res, gate, post, wp, bp, pre, wn, eps):
    """{name: A}: dX, dY, and the terms (one row a token) of dw_pre, db_pre, dw_post, db_post, dgate."""
    out = {}
    g = None
    if dn is not None:
        g, out["dw_pre"], out["db_pre"] = _back(A.of(z), A.of(dn), pre, wn, eps)
    if dz is not None:
        g = A.of(dz) if g is None else g + dz
    out["dX"] = g * res
    if y is not None:
        out["dgate"] = g * norm(A.of(y), post, wp, bp, eps)
        if gate is not None:
            g = g * gate
        out["dY"], out["dw_post"], out["db_post"] = _back(A.of(y), g, post, wp, eps)
    return out
