"""The handles that the binding keeps C structures in: what they may be used for between and
after calls, without a GPU."""
import copy
import gc
import pickle
import weakref

import pytest
import torch

import sparse_kv_long_sfi_gb300 as sfi
from sparse_kv_long_sfi_gb300 import api


@pytest.fixture
def host(monkeypatch):
    """Handles of tensors in host memory (nothing is launched here)."""
    monkeypatch.setattr(api, "_need", lambda t, dtype, name: None)
    monkeypatch.setattr(api, "_on_current_device", lambda t, name: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1, raising=False)


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def _handles():
    return {
        "PagedKV4": sfi.PagedKV4(torch.zeros(5, 2, 1152, dtype=torch.uint8), _i32(3, 4), _i32(3), 2.0, 0.5),
        "CompactKV4": sfi.CompactKV4(torch.zeros(6, 1152, dtype=torch.uint8), torch.zeros(3, dtype=torch.int64),
                                     _i32(3), _i32(3)),
        "Rope": sfi.Rope(torch.arange(8), torch.zeros(8, dtype=torch.uint8), 2, True),
        "Rope without axes": sfi.Rope(torch.arange(8)),
        "PageMap": sfi.PageMap(_i32(3, 4), _i32(3), _i32(9)),
        "PagePools": sfi.PagePools([torch.arange(40).view(5, 8), torch.zeros(5, 8, dtype=torch.int64)]),
    }


def _tensors(h):
    if isinstance(h, sfi.PagePools):
        return h.pools
    return [t for t in vars(h).values() if isinstance(t, torch.Tensor)]


@pytest.mark.parametrize("name", ["PagedKV4", "CompactKV4", "Rope", "Rope without axes", "PageMap", "PagePools"])
def test_handles_are_copied_before_and_after_a_call(host, name):
    for used in (False, True):
        h = _handles()[name]
        if used:
            h.c()
        for copied in (copy.deepcopy(h), pickle.loads(pickle.dumps(h)), copy.copy(h)):
            assert type(copied) is type(h) and len(_tensors(copied)) == len(_tensors(h))
            c, own = copied.c(), h.c()
            assert c is not own
            for a, b in zip(_tensors(copied), _tensors(h)):
                assert torch.equal(a, b)
            first = c._fields_[0][0]
            if isinstance(h, sfi.PagePools):
                assert copied.addresses.tolist() == [t.data_ptr() for t in copied.pools]
                assert getattr(c, first) == copied.addresses.data_ptr()
            else:
                assert getattr(c, first) == _tensors(copied)[0].data_ptr()
            # everything but the addresses is alike
            for f, _ in c._fields_:
                if not isinstance(getattr(c, f), int) or getattr(c, f) < 4096:
                    assert getattr(c, f) == getattr(own, f), f


def test_a_tensor_that_changes_in_place_is_looked_at_again(monkeypatch):
    """A table or pool that gets another shape or other strides where it lies: the structure is made
    anew (the memory's address alone would not say so), and refused where it no longer fits."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1, raising=False)

    def need(t, dtype, name):  # what the binding asks for, but the device
        if t.dtype != dtype or not t.is_contiguous():
            raise ValueError(name)

    monkeypatch.setattr(api, "_need", need)
    kv = sfi.PagedKV4(torch.zeros(5, 2, 1152, dtype=torch.uint8), _i32(4, 4), _i32(4))
    assert kv.c() is kv.c() and kv.c().max_pages_per_req == 4 and kv.c().num_pages == 5
    at = kv.page_table.data_ptr()
    kv.page_table.resize_(4, 3)
    assert kv.page_table.data_ptr() == at
    assert kv.c().max_pages_per_req == 3
    kv.pool.data = kv.pool.data[:3]
    assert kv.pool.data_ptr() == kv.c().pool and kv.c().num_pages == 3
    kv.page_table.resize_(3, 4)  # a row less than there are lengths
    with pytest.raises(ValueError):
        kv.c()
    kv.seq_lens.resize_(3)
    assert kv.c().max_pages_per_req == 4
    kv.page_table.resize_(3, 3)
    assert kv.c() is kv.c()
    kv.page_table.t_()  # the same address and shape
    with pytest.raises(ValueError):
        kv.c()
    pm = sfi.PageMap(_i32(3, 4), _i32(3), _i32(9))
    assert pm.c().num_pages == 9
    pm.ref_count.resize_(7)
    assert pm.c().num_pages == 7
    comp = sfi.CompactKV4(torch.zeros(6, 1152, dtype=torch.uint8), torch.zeros(3, dtype=torch.int64), _i32(3), _i32(3))
    assert comp.c().total_pages == 6
    comp.pool.resize_(4, 1152)
    assert comp.c().total_pages == 4
    rope = sfi.Rope(torch.arange(8), torch.zeros(8, dtype=torch.uint8))
    assert rope.c().rot_dim == 16
    rope.turns.resize_(4)
    with pytest.raises(ValueError):
        rope.c()
    rope.axis.resize_(4)
    assert rope.c().rot_dim == 8


class Fake:
    """As much of a CUDA tensor as the binding looks at, on a device of choice."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.int32, device=0):
        self.t = torch.zeros(*shape, dtype=dtype)
        self.index, self.device = device, torch.device("cuda", device)
        self.dtype, self.shape = dtype, self.t.shape

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        if name in ("data_ptr", "stride", "is_contiguous", "numel", "dim", "nbytes"):
            return getattr(self.t, name)
        raise AttributeError(name)


@pytest.fixture
def two_devices(monkeypatch):
    """Two devices, of which 0 is the current one, and a library that only counts its calls."""
    class State:
        current, launches = 0, []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: State.launches.append(name) or 0

    State.launches = []
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: State.current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    monkeypatch.setattr(api._abi, "lib", Lib)
    return State


BF, F32, U8, I64 = torch.bfloat16, torch.float32, torch.uint8, torch.int64
SHAPE = sfi.AttnShape(4, 2, 64)


def _pools(device):
    t = [Fake(6, 8, dtype=I64, device=device) for _ in range(2)]
    t[0].device = torch.device("cpu")  # where the addresses can go here
    pools = sfi.PagePools(t)
    pools.addresses = Fake(2, dtype=I64, device=device)
    return pools


def _arguments(where=lambda name: 0):
    """Every tensor that the calls take, by name, on the device where(name)."""
    f = lambda name, *s, dtype=torch.int32: Fake(*s, dtype=dtype, device=where(name))  # noqa: E731
    return dict(
        kv=sfi.PagedKV4(f("pool", 6, 2, 1152, dtype=U8), f("page_table", 3, 4), f("seq_lens", 3)),
        bf16=sfi.PagedKV(f("k_pool", 6, 2, 16, 64, dtype=BF), f("v_pool", 6, 2, 16, 64, dtype=BF),
                         f("bf16_table", 3, 4), f("bf16_lens", 3)),
        compact=sfi.CompactKV4(f("blocks", 12, 1152, dtype=U8), f("offset", 3, dtype=I64), f("capacity", 3),
                               f("held", 3)),
        rope=sfi.Rope(f("turns", 32, dtype=I64), f("axis", 32, dtype=U8)),
        map=sfi.PageMap(f("map_table", 3, 4), f("map_lens", 3), f("ref_count", 6)),
        pools=_pools(where("page_pool")),
        q=f("q", 3, 1, 4, 64, dtype=BF), k=f("k", 3, 1, 2, 64, dtype=BF), v=f("v", 3, 1, 2, 64, dtype=BF),
        q_out=f("q_out", 3, 1, 4, 64, dtype=BF), k_out=f("k_out", 3, 1, 2, 64, dtype=BF),
        v_out=f("v_out", 3, 1, 2, 64, dtype=BF), weight=f("weight", 64, dtype=BF), positions=f("positions", 3, 1),
        out=f("out", 3, 1, 4, 64, dtype=F32), lse=f("lse", 3, 1, 4, dtype=F32), scores=f("scores", 3, 2, 64, dtype=F32),
        ws=f("ws", 256, dtype=U8), per=f("per", 3), ids=f("ids", 3), st=f("st", 1), idx=f("idx", 3, 2, 8),
        src=f("src", 2), dst=f("dst", 2), table_out=f("table_out", 3, 4), ref_out=f("ref_out", 6), live=f("live", 1))


CALLS = {
    "qk_norm_rope": (lambda a: sfi.sfi_qk_norm_rope(
        SHAPE, a["rope"], a["q"], a["k"], a["v"], a["q_out"], q_weight=a["weight"], positions=a["positions"],
        new_lens=a["per"], k_out=a["k_out"], kv=a["bf16"], req_ids=a["ids"], dev_status=a["st"]),
        "turns axis q k v q_out weight positions per k_out k_pool v_pool bf16_table bf16_lens ids st"),
    "kv4_append": (lambda a: sfi.sfi_kv4_append(SHAPE, a["kv"], a["k"], a["v"], new_lens=a["per"], req_ids=a["ids"],
                                                dev_status=a["st"]), "pool page_table seq_lens k v per ids st"),
    "kv4_read": (lambda a: sfi.sfi_kv4_read(SHAPE, a["kv"], a["k_out"], a["v_out"], first=a["per"], req_ids=a["ids"],
                                            dev_status=a["st"]), "pool page_table seq_lens k_out v_out per ids st"),
    "kv4_compact_gather": (lambda a: sfi.sfi_kv4_compact_gather(
        SHAPE, a["kv"], a["idx"], a["per"], 4, a["compact"], req_ids=a["ids"], dev_status=a["st"]),
        "pool page_table seq_lens idx per blocks offset capacity held ids st"),
    "kv4_dense_attn": (lambda a: sfi.sfi_kv4_dense_attn(
        SHAPE, a["kv"], 4, 8, a["q"], a["out"], lse=a["lse"], scores=a["scores"], req_ids=a["ids"], workspace=a["ws"],
        dev_status=a["st"]), "pool page_table seq_lens q out lse scores ids ws st"),
    "kv4_fast_attn": (lambda a: sfi.sfi_kv4_fast_attn(
        SHAPE, a["kv"], a["compact"], 4, 8, a["q"], a["out"], lse=a["lse"], req_ids=a["ids"], workspace=a["ws"],
        dev_status=a["st"]), "pool page_table seq_lens blocks offset capacity held q out lse ids ws st"),
    "page_copy": (lambda a: sfi.sfi_page_copy(a["pools"], a["src"], a["dst"], dev_status=a["st"]),
                  "page_pool src dst st"),
    "page_fork": (lambda a: sfi.sfi_page_fork(a["map"], a["src"], a["dst"], a["src"], dev_status=a["st"]),
                  "map_table map_lens ref_count src dst st"),
    "page_reserve": (lambda a: sfi.sfi_page_reserve(a["map"], a["pools"], a["per"], a["ids"], workspace=a["ws"],
                                                    dev_status=a["st"]),
                     "page_pool map_table map_lens ref_count per ids ws st"),
    "page_free": (lambda a: sfi.sfi_page_free(a["map"], a["ids"], dev_status=a["st"]),
                  "map_table map_lens ref_count ids st"),
    "page_compact": (lambda a: sfi.sfi_page_compact(a["map"], a["pools"], a["table_out"], a["ref_out"], a["live"],
                                                    workspace=a["ws"], dev_status=a["st"]),
                     "page_pool map_table map_lens ref_count table_out ref_out live ws st"),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_no_tensor_of_another_device_reaches_a_launch(two_devices, name):
    call, tensors = CALLS[name]
    call(_arguments())
    assert two_devices.launches == ["sfi_" + name]
    for t in tensors.split():
        with pytest.raises(ValueError, match="not on the current device"):
            call(_arguments(lambda n: int(n == t)))
            pytest.fail(f"{t} of device 1 was taken")
    assert two_devices.launches == ["sfi_" + name]


@pytest.mark.parametrize("name", list(CALLS))
def test_the_device_is_looked_at_in_every_call(two_devices, name):
    """A handle that was used under its own device is refused under another one, and taken again."""
    call, a = CALLS[name][0], _arguments()
    call(a)
    two_devices.current = 1
    for _ in range(2):
        with pytest.raises(ValueError, match="not on the current device"):
            call(a)
    # all else on the new device: the handles alone say no
    handles = ("kv", "bf16", "compact", "rope", "map", "pools")
    b = {**_arguments(lambda n: 1), **{k: a[k] for k in handles}}
    with pytest.raises(ValueError, match="not on the current device"):
        call(b)
    two_devices.current = 0
    call(a)
    assert two_devices.launches == ["sfi_" + name] * 2


def test_pools_that_moved_are_refused(host):
    """The device array of the pools' addresses is written once: a pool whose memory was replaced
    must not be copied at the old place."""
    pools = [torch.arange(40).view(5, 8) for _ in range(3)]
    pp = sfi.PagePools(pools)
    assert pp.c().num_pages == 5 and pp.c() is pp.c()
    keep = pools[1].data
    pools[1].data = torch.zeros(5, 8, dtype=torch.int64)
    with pytest.raises(ValueError, match="other memory"):
        pp.c()
    pools[1].data = keep
    assert pp.c().num_pages == 5
    pools[0].resize_(500, 8)
    with pytest.raises(ValueError, match="other memory"):
        pp.c()


def test_the_norm_takes_a_table_with_a_row_for_each_request(two_devices):
    """qk_norm_rope indexes the page table by request: one with fewer rows than q, k and v have
    requests (or with more, or not a table) is refused before a launch, as PagedKV4 refuses it."""
    call, a = CALLS["qk_norm_rope"][0], _arguments()
    for table in (Fake(2, 4), Fake(1, 4), Fake(4, 4), Fake(3), Fake(3, 4, 1), Fake(12)):
        a["bf16"].page_table = table
        with pytest.raises(ValueError):
            call(a)
    a["bf16"].page_table = Fake(3, 5)
    for lens in (Fake(2), Fake(4)):
        a["bf16"].seq_lens = lens
        with pytest.raises(ValueError):
            call(a)
    assert two_devices.launches == []
    a["bf16"].seq_lens = Fake(3)
    call(a)
    assert two_devices.launches == ["sfi_qk_norm_rope"]


def test_a_handle_lets_go_of_a_replaced_tensor(host):
    """What a call has kept of a handle's tensors does not outlive their place in it: a pool that is
    replaced, or set to None to make room, is freed at once."""
    kv = _handles()["PagedKV4"]
    kv.c()
    old = weakref.ref(kv.pool)
    kv.pool = None
    gc.collect()
    assert old() is None
    with pytest.raises(AttributeError):
        kv.c()
    kv.pool = torch.zeros(7, 2, 1152, dtype=torch.uint8)
    assert kv.c().num_pages == 7
    old = weakref.ref(kv.page_table)
    kv.page_table = _i32(3, 6)
    gc.collect()
    assert old() is None and kv.c().max_pages_per_req == 6
