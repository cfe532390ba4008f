"""The serving step's Python calls refuse tensors of several devices, on the host: tensors without memory stand for those of
GPUs that this machine need not have (nothing reads or launches anything before the refusal)."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def w():
    from weight_only_int4_02_gb300 import build
    build.build()
    from weight_only_int4_02_gb300 import w4a16
    return w4a16


class Elsewhere(torch.Tensor):
    """A tensor's type, shape and device alone."""

    @staticmethod
    def __new__(cls, dtype, *shape, device="cuda:0"):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device=device)

    @classmethod
    def __torch_dispatch__(cls, f, types, args=(), kwargs=None):
        raise AssertionError("%s was called" % f)


def test_tensors_of_two_devices_are_refused(w):
    t = Elsewhere
    i32, i64, f16, f32, u8 = torch.int32, torch.int64, torch.float16, torch.float32, torch.uint8
    cache = t(u8, 3, 2, 1, 16 * 70)
    kv = t(f16, 5, 2, 64)
    calls = [(lambda *a: w.kv4_tables(*a[:4], 16, 5, taken=a[4]), [t(i32, 2), t(i32, 2), t(i32, 4), t(i32, 2, 3), t(i32, 1)]),
             (lambda *a: w.kv4_append(*a, 16), [kv, kv, t(i64, 5), cache]),
             (lambda *a: w.kv4_read(*a, 16), [cache, t(i64, 5)]),
             (lambda *a: w.kv4_attention(*a[:5], 16, 1, out=a[5], workspace=a[6]),
              [t(f16, 5, 4, 64), cache, t(i32, 2, 3), t(i32, 2), t(i32, 3), t(f16, 5, 4, 64), t(u8, 4096)]),
             (w.sample, [t(f32, 4, 9), t(f32, 4), t(f32, 4), t(i32, 4), t(f32, 4), t(f32, 4)])]
    for call, args in calls:
        for i, a in enumerate(args):
            mixed = list(args)
            mixed[i] = t(a.dtype, *a.shape, device="cuda:1")
            with pytest.raises(w.W4A16Error, match="one device") as e:
                call(*mixed)
            assert e.value.status == w.ERR_INVALID_ARG
