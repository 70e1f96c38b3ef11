"""CPU checks of the operators around a speculative decode step: every call
with a bad argument is refused with its status before a device is looked for,
and a good one without a device says so.  The addresses are never
dereferenced."""
import ctypes as C

import pytest

from fp4_compressed_kv_b200 import synth

A = 0x10000  # an aligned address
OK, INVALID, CAPACITY, NO_DEVICE = 0, 1, 2, 6


@pytest.fixture(scope="module")
def lib():
    from fp4_compressed_kv_b200 import build, kvc
    build.build()
    return kvc


def _calls(lib):
    """name -> (function, good arguments by name)."""
    so = lib.lib()
    cfg = lib.config_for(synth.WORKLOADS["mla32k"])
    cache = lib.CacheStruct(A, A, A, 2, 100)
    d = cfg.latent_dim + cfg.rope_dim
    return {
        "norm_rope": (so.kvc_norm_rope, dict(
            cfg=cfg, n_rows=5, q=A, q_stride=cfg.n_heads * d, q_gain=A, q_norm=2, q_out=A, k=A,
            k_stride=d, k_gain=A, k_norm=1, k_out=A, positions=A, inv_freq=A, eps=1e-6, layout=0,
            status=None, stream=None)),
        "unpack": (so.kvc_unpack, dict(cfg=cfg, cache=cache, idx=None, first=0, n=100, rows=A,
                                       status=None, stream=None)),
        "unpack_fp8": (so.kvc_unpack_window_fp8, dict(cfg=cfg, codes=A, scales=A, n_rows=7, rows=A,
                                                      stream=None)),
        "tree": (so.kvc_tree_decode_attn, dict(
            cfg=cfg, n_nodes=4, q=A, cache=cache, topk=A, shared=0, window=A, window_len=128,
            window_lens=None, draft=A, parents=A, out=A, lse=None, status=None, stream=None)),
        "verify": (so.kvc_verify_tree, dict(
            batch=2, n_nodes=4, vocab=1000, dtype=0, p=A, p_stride=1000, q=A, q_stride=1000,
            tokens=A, parents=A, u=A, v=A, path=A, n_path=A, next=A, status=None, stream=None))}


def _call(fn, args, **change):
    a = dict(args, **change)
    return fn(*[C.byref(x) if isinstance(x, C.Structure) else x for x in a.values()])


BAD = {
    "norm_rope": [(dict(n_rows=-1), INVALID), (dict(q_norm=3), INVALID), (dict(k_norm=-1), INVALID),
                  (dict(layout=2), INVALID), (dict(eps=-1.0), INVALID),
                  (dict(eps=float("nan")), INVALID), (dict(q=None, k=None), INVALID),
                  (dict(q_out=None), INVALID), (dict(k_out=None), INVALID),
                  (dict(positions=None), INVALID), (dict(inv_freq=None), INVALID),
                  (dict(q_stride=64 * 576 - 8), INVALID), (dict(q_stride=64 * 576 + 4), INVALID),
                  (dict(k_stride=575), INVALID), (dict(q=A + 8), INVALID), (dict(k_out=A + 2), INVALID),
                  (dict(q_gain=A + 4), INVALID), (dict(q_stride=64 * 576 + 8), INVALID),
                  (dict(k_stride=584), INVALID)],  # (in place only where rows coincide)
    "unpack": [(dict(first=-1), INVALID), (dict(first=1), INVALID), (dict(n=-1), INVALID),
               (dict(rows=None), INVALID), (dict(rows=A + 8), INVALID), (dict(idx=A + 2), INVALID)],
    "unpack_fp8": [(dict(n_rows=-1), INVALID), (dict(codes=None), INVALID),
                   (dict(codes=A + 4), INVALID), (dict(scales=A + 2), INVALID),
                   (dict(rows=A + 8), INVALID)],
    "tree": [(dict(n_nodes=-1), INVALID), (dict(n_nodes=257), CAPACITY), (dict(shared=2), INVALID),
             (dict(window_len=129), INVALID), (dict(window_len=-1), INVALID), (dict(q=None), INVALID),
             (dict(topk=None), INVALID), (dict(window=None), INVALID), (dict(draft=None), INVALID),
             (dict(parents=None), INVALID), (dict(out=None), INVALID), (dict(q=A + 8), INVALID),
             (dict(draft=A + 8), INVALID), (dict(out=A + 8), INVALID), (dict(parents=A + 2), INVALID),
             (dict(lse=A + 2), INVALID), (dict(window_lens=A + 1), INVALID)],
    "verify": [(dict(batch=-1), INVALID), (dict(n_nodes=0), INVALID), (dict(n_nodes=257), CAPACITY),
               (dict(vocab=0), INVALID), (dict(vocab=4_194_305, p_stride=1 << 23, q_stride=1 << 23),
                                          CAPACITY),
               (dict(batch=65_536), CAPACITY), (dict(dtype=2), INVALID), (dict(p=None), INVALID),
               (dict(p_stride=999), INVALID), (dict(q_stride=999), INVALID), (dict(p=A + 2), INVALID),
               (dict(u=None), INVALID), (dict(v=None), INVALID), (dict(path=None), INVALID),
               (dict(n_path=None), INVALID), (dict(next=None), INVALID), (dict(tokens=A + 2), INVALID)],
}


@pytest.mark.parametrize("name", BAD)
def test_refused_before_any_device(lib, name):
    fn, good = _calls(lib)[name]
    for change, status in BAD[name]:
        assert _call(fn, good, **change) == status, change
    if "cfg" in good:
        bad = lib.config_for(synth.WORKLOADS["mla32k"])
        bad.group = 48
        assert _call(fn, good, cfg=bad) == INVALID
    if "cache" in good:
        for fields in ((None, A, A, 2, 100), (A, A, None, 2, 100), (A, A, A, -1, 100),
                       (A, A, A, 2, -1), (A + 8, A, A, 2, 100), (A, A, A + 2, 2, 100)):
            assert _call(fn, good, cache=lib.CacheStruct(*fields)) == INVALID
        assert _call(fn, good, cache=lib.CacheStruct(A, A, A, 65_536, 100)) == CAPACITY


def test_nothing_to_do_needs_no_device(lib):
    calls = _calls(lib)
    none = lib.CacheStruct(A, None, A, 0, 100)
    for name, change in (("norm_rope", dict(n_rows=0)), ("unpack", dict(n=0)),
                         ("unpack", dict(cache=none)), ("unpack_fp8", dict(n_rows=0)),
                         ("tree", dict(n_nodes=0)), ("tree", dict(cache=none)),
                         ("verify", dict(batch=0))):
        assert _call(*calls[name], **change) == OK


def test_without_a_device(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    for name, (fn, good) in _calls(lib).items():
        assert _call(fn, good) == NO_DEVICE, name
        if name == "norm_rope":
            # keys alone; RoPE-free rows need no frequencies; rows in place
            assert _call(fn, good, q=None, q_out=None, q_gain=None) == NO_DEVICE
        if name in ("unpack", "tree"):
            assert _call(fn, good, cache=lib.CacheStruct(A, None, A, 2, 100)) == NO_DEVICE


def test_unpack_counts_its_rows_in_32_bits(lib):
    """A row number and a tile behind it stay below 2^31; more rows are refused."""
    fn, args = _calls(lib)["unpack"]
    for n in (2**31 - 1, 2**31 - 2**16 + 1):
        assert _call(fn, args, idx=A, n=n) == CAPACITY


def test_a_norm_without_a_name_is_refused_as_such(lib, monkeypatch):
    """The wrapper leaves an unknown norm to the library's own check."""
    import torch
    cfg = lib.make_config(64, 16, 16, lib.SCALE_UE4M3, 32, 8, 16, 8, 0.1, lib.BF16)
    monkeypatch.setattr(lib, "_here", lambda stream: (-1, 0))  # tensors of the host stand in
    k, out = (torch.zeros(3, 80, dtype=torch.bfloat16) for _ in range(2))
    pos, freq = torch.zeros(3, dtype=torch.int32), torch.zeros(8)
    for norm in (3, -1):
        with pytest.raises(lib.KvcError):
            lib.norm_rope(cfg, None, k, pos, freq, None, out, k_norm=norm)


def test_a_cache_of_another_layout_or_device_is_refused(lib, monkeypatch):
    """The kernels step through the records by the call's record size: a cache
    whose records another configuration laid out, or whose buffers are not on
    the current device, does not reach the library."""
    import torch

    class Reached(Exception):
        pass

    class Stub:  # the library, but nothing of it that would launch
        kvc_record_bytes = lib.lib().kvc_record_bytes
        kvc_idx_row_bytes = lib.lib().kvc_idx_row_bytes

        def __getattr__(self, name):
            def call(*args):
                raise Reached
            return call

    def config(group=32, fmt=lib.SCALE_UE4M3, latent=64, rope=16, heads=8):
        return lib.make_config(latent, rope, group, fmt, 32, 8, 16, heads, 0.1, lib.F32)

    here = [-1]  # tensors of the host stand in
    stub = Stub()
    monkeypatch.setattr(lib, "_here", lambda stream: (here[0], 0))
    monkeypatch.setattr(lib, "_lib", lambda: stub)
    cfg = config()
    i32 = dict(dtype=torch.int32)
    rows, q = torch.zeros(2, 5, 80), torch.zeros(3, 2, 8, 80)
    topk, win, draft = torch.zeros(3, 2, 8, **i32), torch.zeros(2, 16, 80), torch.zeros(3, 2, 80)
    par, out = torch.zeros(3, 2, **i32), torch.zeros(3, 2, 8, 64)

    def calls(c, cache):
        return (lambda: lib.unpack(c, cache, rows),
                lambda: lib.tree_decode_attn(c, q, cache, topk, win, 16, draft, par, out))

    good = lib.Cache(cfg, 2, 20, device="cpu")
    for call in calls(cfg, good) + calls(config(heads=8), good):
        with pytest.raises(Reached):
            call()
    # a longer record, a shorter one, and one of the same size that means something else
    others = [config(group=8), config(group=64, fmt=lib.SCALE_F32), config(group=16),
              config(latent=48, rope=32, group=16)]
    assert lib.record_bytes(others[2]) == lib.record_bytes(cfg) != lib.record_bytes(others[0])
    for other in others:
        for call in calls(cfg, lib.Cache(other, 2, 20, device="cpu")):
            with pytest.raises(ValueError):
                call()
    # a configuration changed behind its cache, and buffers changed behind it
    changed = config()
    cache = lib.Cache(changed, 2, 20, device="cpu")
    changed.scale_fmt = lib.SCALE_F32
    for call in calls(changed, cache):
        with pytest.raises(ValueError):
            call()
    for name, t in (("records", good.records[:1]), ("records", good.records[:, ::2]),
                    ("n_entries", good.n_entries.long()), ("n_entries", good.n_entries[:1])):
        cache = lib.Cache(cfg, 2, 20, device="cpu")
        setattr(cache, name, t)
        for call in calls(cfg, cache):
            with pytest.raises(ValueError):
                call()
    # buffers on another device than the current one
    here[0] = 0
    with pytest.raises(ValueError):
        lib.unpack(cfg, good, rows)
    # an invalid configuration is left to the library's own check
    here[0] = -1
    for call in calls(config(group=48), good):
        with pytest.raises(Reached):
            call()
