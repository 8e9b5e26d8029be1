"""CPU tests of the paged cache's Python wrappers: index tensors of another type
or layout than the entry points read are refused before the call, and views that
they do read pass."""
import pytest
import torch

I32, I64, BF = torch.int32, torch.int64, torch.bfloat16


@pytest.fixture
def calls(qmm, monkeypatch):
    """The arguments that reach the library."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            def entry(*args):
                seen.append((name, args))
                return qmm.QMM_OK
            return entry

    monkeypatch.setattr(qmm, "lib", Lib())
    monkeypatch.setattr(qmm, "_raw_stream", lambda device: 0)
    return seen


def z(*shape, dtype=I32):
    return torch.zeros(shape, dtype=dtype)


def plan_args(**over):
    a = dict(ctx=z(4), new=z(4), free=z(9), table=z(4, 5), page=16, slots=z(6, dtype=I64), positions=z(6),
             cu_new=z(5), pages_taken=z(1), parents=z(6), mask=z(6, 2), dev_status=z(1))
    a.update(over)
    return a


def plan(qmm, a):
    return qmm.kv_plan(a["ctx"], a["new"], a["free"], a["table"], a["page"], a["slots"], a["positions"],
                       cu_new=a["cu_new"], pages_taken=a["pages_taken"], parents=a["parents"], mask=a["mask"],
                       dev_status=a["dev_status"])


@pytest.mark.parametrize("name,size", [("ctx", 4), ("new", 4), ("free", 9), ("slots", 6), ("positions", 6),
                                       ("cu_new", 5), ("pages_taken", 1), ("parents", 6), ("dev_status", 1)])
def test_plan_vectors(qmm, calls, name, size):
    other = I32 if name == "slots" else I64
    own = I64 if name == "slots" else I32
    with pytest.raises(ValueError, match="contiguous"):
        plan(qmm, plan_args(**{name: z(size, dtype=other)}))
    with pytest.raises(ValueError, match="contiguous"):
        plan(qmm, plan_args(**{name: z(size, dtype=torch.float32)}))
    if size > 1:                                  # one element has no order
        with pytest.raises(ValueError, match="contiguous"):
            plan(qmm, plan_args(**{name: z(size, 3, dtype=own)[:, 0]}))
    assert not calls
    plan(qmm, plan_args(**{name: z(size + 3, dtype=own)[1:1 + size]}))   # a plain slice
    assert len(calls) == 1


def test_plan_tables(qmm, calls):
    for bad in (dict(table=z(4, 5, dtype=I64)), dict(table=z(5, 4).t()), dict(table=z(4, 10)[:, ::2]),
                dict(mask=z(6, 2, dtype=I64)), dict(mask=z(2, 6).t()), dict(mask=z(6, 4)[:, ::2])):
        with pytest.raises(ValueError, match="contiguous rows"):
            plan(qmm, plan_args(**bad))
    assert not calls
    plan(qmm, plan_args(table=z(4, 9)[:, 2:7], mask=z(6, 7)[:, 3:5]))
    (_, a), = calls
    assert a[6:8] == (9, 5) and a[11:14] == (7, 2, 6)
    calls.clear()
    plan(qmm, plan_args(mask=z(6, 2).view(torch.uint32)))
    assert len(calls) == 1
    calls.clear()
    one = dict(ctx=z(1), new=z(1), table=z(5, 7).t()[:1], cu_new=z(2), slots=z(1, dtype=I64), positions=z(1),
               parents=z(1), mask=z(1, 2))
    with pytest.raises(ValueError, match="contiguous rows"):
        plan(qmm, plan_args(**one))
    one["table"] = torch.as_strided(z(8), (1, 5), (1, 1))   # one row: its stride says nothing
    plan(qmm, plan_args(**one))
    assert calls[0][1][6:8] == (5, 5)


def test_append(qmm, calls):
    k = z(2, 4, 2, 64, dtype=BF)
    rows = torch.zeros((3, 2, 64))
    for bad in (z(3), z(3, dtype=torch.int16), z(3, 2, dtype=I64)[:, 0]):
        with pytest.raises(ValueError, match="contiguous"):
            qmm.kv_append(rows, rows, bad, k, k)
    with pytest.raises(ValueError, match="contiguous"):
        qmm.kv_append(rows, rows, z(3, dtype=I64), k, k, dev_status=z(1, dtype=torch.uint8))
    assert not calls
    qmm.kv_append(rows, rows, z(5, dtype=I64)[1:4], k, k, dev_status=z(1))
    assert len(calls) == 1


def test_attention(qmm, calls):
    k, q = z(2, 4, 2, 64, dtype=BF), z(3, 4, 64, dtype=BF)
    base = dict(t=z(2, 2), ctx=z(2), cu=z(3), mask=z(3, 1), status=z(1), ws=z(1 << 20, dtype=torch.uint8), max_new=3)

    def call(**over):
        a = {**base, **over}
        return qmm.tree_attention(q, k, k, a["t"], a["ctx"], a["cu"], a["max_new"], mask=a["mask"],
                                  workspace=a["ws"], dev_status=a["status"])

    for bad in (dict(ctx=z(2, dtype=I64)), dict(ctx=z(2, 3)[:, 0]), dict(cu=z(3, dtype=I64)), dict(cu=z(6)[::2]),
                dict(status=z(1, dtype=torch.int16)), dict(t=z(2, 2, dtype=I64)), dict(t=z(2, 2).t()),
                dict(t=z(2, 4)[:, ::2]), dict(mask=z(3, 1, dtype=I64)), dict(mask=z(3, 4)[:, ::2], max_new=40)):
        with pytest.raises(ValueError, match="contiguous"):
            call(**bad)
    # a view of too few words, in a buffer of enough
    with pytest.raises(ValueError, match="agree"):
        call(mask=z(3, 4)[:, :1], max_new=33)
    assert not calls
    call(mask=z(3, 4)[:, 1:3], max_new=33)
    call(mask=None, t=z(2, 6)[:, 1:3])
    call(mask=z(3, 1).view(torch.uint32))
    assert len(calls) == 3 and calls[0][1][15] == 4 and calls[1][1][7:9] == (6, 2)
