"""Host side of the serving operators, next to test_serving_cpu.py: the cache's tensors, the build, sizes and strides."""

import pytest
import torch


def test_cache_tensors_change_in_place_only():
    """`cache.lens += 1` counts once and does not raise; another tensor is refused before anything has changed."""
    from linear_attention_nats_gb300.paged import PagedCache

    names = ("k_pages", "v_pages", "table", "lens", "weight", "err")
    c = PagedCache.__new__(PagedCache)
    c._t = tuple(torch.zeros(2, dtype=torch.int32) for _ in names)
    for name, t in zip(names, c._t):
        assert getattr(c, name) is t
        setattr(c, name, t)
        with pytest.raises(AttributeError):
            setattr(c, name, t.clone())
    c.lens += 1
    assert c.lens is c._t[3] and c.lens.tolist() == [1, 1]
    with pytest.raises(AttributeError):
        c.lens = c.lens + 1
    assert c.lens.tolist() == [1, 1]


# --------------------------------------------------------------- the build

@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """The build with its files in a folder of their own and compilers that only write what they are told to; returns
    (build, the commands run, the names of programs that fail)."""
    import os
    import types

    from linear_attention_nats_gb300 import build as b

    for name, path in (("BUILD", "_build"), ("LIB", "libnats.so"), ("BINDING", "_operators.so"), ("STAMP", "_build/binding.txt")):
        monkeypatch.setattr(b, name, str(tmp_path / path), raising=False)
    ran, failing = [], set()

    def run(cmd, **kw):
        name = os.path.basename(cmd[0])
        ran.append(name)
        if name in failing:
            return types.SimpleNamespace(returncode=1, stdout="", stderr="no headers")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setenv("CXX", "g++")
    return b, ran, failing


def test_the_library_is_linked_where_its_binding_cannot_be(sandbox):
    import os

    b, ran, failing = sandbox
    failing.add("g++")
    with pytest.raises(RuntimeError, match="binding"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING) and not b.up_to_date()
    ran.clear()
    with pytest.raises(RuntimeError, match="binding"):
        b.build()
    assert ran == ["g++"]  # nothing of the library again
    failing.clear()
    b.build()
    assert os.path.exists(b.BINDING) and b.up_to_date()


def test_the_binding_is_built_again_for_another_python_or_torch(sandbox, monkeypatch):
    import importlib.metadata

    b, ran, _ = sandbox
    b.build()
    assert b.up_to_date() and "nvcc" in ran
    ran.clear()
    b.build()
    assert ran == []
    version = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda n: "0.0" if n == "torch" else version(n))
    assert not b.up_to_date()
    b.build()
    assert ran == ["g++"] and b.up_to_date()
    monkeypatch.setattr(b.sys, "version", "4.0")
    b.build()
    assert ran == ["g++", "g++"]


# ----------------------------------------------------------------- strides

def test_decode_takes_any_stride_of_one_sequence_or_head():
    """A stride between one row and nothing says nothing (torch leaves what it likes there, .contiguous() too): the
    call goes on to its next check, a workspace that is too small."""
    from linear_attention_nats_gb300 import build as b

    b.build()
    from linear_attention_nats_gb300 import _native as nat

    A = 0x10000000

    def call(B, Hq, qb, qh):
        c = nat.PagedCache(A, A, A, A, A, A, 8, 16, 1, 64, B, 4, 0)
        return nat.lib.nats_paged_decode(c, Hq, 0.0, A, qb, qh, A, None, 0, A, 0, None)

    assert call(1, 4, 259, 64) == 5 and call(2, 4, 259, 64) == 4
    assert call(3, 1, 64, 5) == 5 and call(3, 2, 64, 5) == 4
    assert call(1, 1, 3, 5) == 5


# ---------------------------------------------------------------- workspace

def test_weights_workspace_is_the_pools_where_tables_are_long():
    """An accumulating call has no page in its table twice, so that scores of every slot of the pool are enough."""
    from linear_attention_nats_gb300 import build as b

    b.build()
    from linear_attention_nats_gb300 import _native as nat

    A = 0x10000000

    def scores(B, Hq, n_pages, max_pages):
        c = nat.PagedCache(A, A, A, A, A, A, n_pages, 64, 8, 128, B, max_pages, 0)
        size = nat.lib.nats_paged_decode_workspace_size
        return size(c, Hq, 1) - size(c, Hq, 0) if size(c, Hq, 1) else None

    pool = 4 * 4096 * 64 * 32
    assert scores(32, 32, 4096, 2048) == pool
    assert scores(32, 32, 4096, 128) == pool  # as many slots as the pool
    assert scores(32, 32, 65536, 128) == pool  # a part of a larger pool
    # 2^41 slots and heads in the table, 2^27 in the pool; and too many of both
    assert scores(1024, 128, 16384, 1 << 18) == 4 * 16384 * 64 * 128
    assert scores(1024, 4096 * 8, 1 << 21, 1 << 18) is None
