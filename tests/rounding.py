"""Values with a bound of the rounding error that a computation in fp32 leaves in them (running error
analysis, first order): every operation adds half a step of its result, sums over n terms n of them,
whatever their order, and the library's functions their documented errors."""

import numpy as np

U = 2.0 ** -24  # half an fp32 step, relative
LIBRARY = 4 * U  # exp, rsqrt: at most two steps


class Rounded:
    __array_ufunc__ = None  # arrays leave operations with one to it

    def __init__(self, value, error=0.0):
        self.v = np.asarray(value, dtype=np.float64)
        self.e = np.broadcast_to(np.asarray(error, dtype=np.float64), self.v.shape)

    @staticmethod
    def of(a):
        return a if isinstance(a, Rounded) else Rounded(a)

    def _new(self, v, e, step=U):
        return Rounded(v, e + step * np.abs(v))

    def __add__(self, o):
        o = Rounded.of(o)
        return self._new(self.v + o.v, self.e + o.e)

    __radd__ = __add__

    def __neg__(self):
        return Rounded(-self.v, self.e)

    def __sub__(self, o):
        return self + (-Rounded.of(o))

    def __rsub__(self, o):
        return Rounded.of(o) + (-self)

    def __mul__(self, o):
        o = Rounded.of(o)
        return self._new(self.v * o.v, np.abs(self.v) * o.e + np.abs(o.v) * self.e)

    __rmul__ = __mul__

    def __truediv__(self, o):
        o = Rounded.of(o)
        v = self.v / o.v
        return self._new(v, self.e / np.abs(o.v) + np.abs(v / o.v) * o.e)

    def __rtruediv__(self, o):
        return Rounded.of(o) / self

    def sum(self, axis, keepdims=False):
        n = self.v.shape[axis]
        return Rounded(self.v.sum(axis, keepdims=keepdims),
                       (self.e + n * U * np.abs(self.v)).sum(axis, keepdims=keepdims))

    def rsqrt(self):
        v = 1 / np.sqrt(self.v)
        return self._new(v, 0.5 * v / self.v * self.e, LIBRARY)

    def exp(self):
        v = np.exp(self.v)
        return self._new(v, v * self.e, LIBRARY)

    def sigmoid(self):
        """1 / (1 + exp(-v)).  Below -80, where exp(-v) may be infinite in fp32 and this 0: off by its own
        size at most, which an error e of v makes exp(e) times as large."""
        low = self.v < -80
        r = 1.0 / (1.0 + (-Rounded(np.where(low, 0.0, self.v), np.where(low, 0.0, self.e))).exp())
        own = np.exp(np.where(low, self.v, 0.0))
        return Rounded(np.where(low, own, r.v),
                       np.where(low, own * np.exp(np.minimum(self.e, 600.0)), r.e))

    def close(self, got, last=U, what=""):
        """|got - value| within the bound and a last rounding of relative size `last`."""
        got = np.asarray(got, dtype=np.float64)
        bound = self.e * (1 + last) + last * np.abs(self.v) + 1e-37
        bad = ~(np.abs(got - self.v) <= bound)
        assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.abs(got - self.v) / bound)))
