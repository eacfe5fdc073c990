"""Checks of the paged-cache and beam-search calls that need no GPU: what the
binding and the library refuse before anything runs on a device."""
import sys
import types

import pytest

import bwd_step_b200
from bwd_step_b200 import Model, _lib
from bwd_step_b200.generate import PagedCache, beam_search

torch = pytest.importorskip("torch")


def _model():
    """A model without a handle: the library refuses it, the binding checks as ever."""
    m = object.__new__(Model)
    m._h, m.device, m.precision = None, 0, "bf16"
    m._handle, m._bf16 = None, True
    m.cfg = types.SimpleNamespace(n_layer=2, n_head=4, n_kv_head=1, head_dim=64, vocab=512)
    return m


def test_status_strings_of_the_paged_calls():
    L = bwd_step_b200.lib()
    for code in (_lib.NC_ERR_OUT_OF_PAGES, _lib.NC_ERR_BAD_LENGTH, _lib.NC_ERR_BAD_PAGE):
        assert L.nc_status_string(code) != L.nc_status_string(-99)


def test_the_library_refuses_a_null_model():
    L, n = bwd_step_b200.lib(), None
    bad = _lib.NC_ERR_INVALID_ARG
    assert L.nc_page_plan(n, 1, 16, 1, 1, 1, *[n] * 11) == bad
    assert L.nc_paged_attention(n, n, 1, 1, 0, n, n, n, n, 1, 16, 1, n, n, n, n, 0, n) == bad
    assert L.nc_paged_forward(n, n, 1, 1, 0, n, n, n, n, n, 1, 16, 1, n, n, n, n, 0, n) == bad
    assert L.nc_beam_select(n, n, 1, 1, n, n, -1, n, n, n, n, n) == bad
    assert L.nc_beam_reorder(n, n, 1, 1, 1, n, 0, 1, n) == bad
    assert L.nc_beam_reorder_paged(n, n, 1, 1, 1, 16, n, n, 1, n, n, n) == bad
    assert L.nc_paged_kv_bytes(n, 1, 16) == L.nc_paged_workspace_bytes(n, 1, 1) == 0
    assert L.nc_paged_attention_workspace_bytes(n, 1, 1) == 0


def test_addresses_are_checked():
    m = _model()
    z, s, i = torch.zeros(2, 3, 512, dtype=torch.bfloat16), torch.zeros(2, 3), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="device memory"):
        m.beam_select(z, s, s, i, i, stream=0)
    with pytest.raises(TypeError, match="expected torch.bfloat16, got torch.float32"):
        m.beam_select(z.float(), s, s, i, i, stream=0)
    with pytest.raises(ValueError, match="contiguous"):
        m.beam_select(torch.zeros(2, 512, 3, dtype=torch.bfloat16).transpose(1, 2), s, s, i, i, stream=0)
    with pytest.raises(TypeError, match="must be a tensor"):
        m.beam_select(z, s, s, [0], i, stream=0)
    with pytest.raises(ValueError, match="eos is out of range"):
        m.beam_select(z, s, s, i, i, eos=1 << 40, stream=0)
    with pytest.raises(ValueError, match=r"tokens must be \[2, 3\], got \[6\]"):
        m.beam_select(z, s, s, i.view(-1), i, stream=0)


def test_shapes_are_checked_before_addresses():
    m = _model()
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    h = lambda *n: torch.zeros(*n, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError, match="cu_rows"):
        m.page_plan(16, i(2), i(2), i(2, 1), i(8), i(1), i(2), i(2), i(4), i(4), stream=0)
    with pytest.raises(ValueError, match="block_table"):
        m.page_plan(16, i(2), i(2), i(3, 1), i(8), i(1), i(3), i(2), i(4), i(4), stream=0)
    with pytest.raises(ValueError, match="release"):
        m.page_plan(16, i(2), i(2), i(2, 1), i(8), i(1), i(3), i(2), i(4), i(4), release=i(3), stream=0)
    args = dict(qkv=h(4, 384), cu_rows=i(3), kv_len=i(2), slots=i(4), block_table=i(2, 5), k_pages=h(9, 16, 1, 64),
                v_pages=h(9, 16, 1, 64), o=h(4, 256), workspace=torch.zeros(256, dtype=torch.uint8))
    for name, bad in (("qkv", h(4, 383)), ("cu_rows", i(2)), ("slots", i(5)), ("block_table", i(3, 5)), ("o", h(3, 256)),
                      ("k_pages", h(9, 16, 2, 64)), ("v_pages", h(8, 16, 1, 64))):
        with pytest.raises(ValueError, match=name):
            m.paged_attention(**{**args, name: bad}, stream=0)
    with pytest.raises(ValueError, match="logits"):
        m.beam_select(h(2, 3, 511), torch.zeros(2, 3), torch.zeros(2, 3), i(2, 3), i(2, 3), stream=0)
    with pytest.raises(ValueError, match="together"):
        m.beam_select(h(2, 3, 512), torch.zeros(2, 3), torch.zeros(2, 3), i(2, 3), i(2, 3), finished=i(2, 3), stream=0)
    with pytest.raises(ValueError, match="parents"):
        m.beam_reorder_paged(h(2, 2, 9, 16, 1, 64), i(4), i(4, 5), i(4), i(4), stream=0)
    with pytest.raises(ValueError, match="block_table"):
        m.beam_reorder_paged(h(2, 2, 9, 16, 1, 64), i(2, 2), i(3, 5), i(4), i(4), stream=0)


def test_searches_that_cannot_run_are_refused():
    m = _model()
    for prompts, beams, new in (([], 2, 1), ([[1], []], 2, 1), ([[1]], 2, 0), ([[1]], 0, 1), ([[1]], 33, 1)):
        with pytest.raises(ValueError):
            beam_search(m, None, prompts, beams, new)


def test_a_step_of_more_rows_than_the_cache_was_made_for_is_refused():
    """Before anything is planned: the cache would claim positions that no forward can write."""
    calls = []
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    c = object.__new__(PagedCache)
    c.model = types.SimpleNamespace(page_plan=lambda *a, **kw: calls.append(a))
    c.page_size, c.n_req = 16, 2
    c.kv_len, c.cu_rows, c.block_table, c.free_pages, c.free_count = i(2), i(3), i(4).view(2, 2), i(4), i(1)
    c._positions, c._slots = i(8), i(8)
    for rows in (9, 0, -1):
        with pytest.raises(ValueError, match="rows"):
            c.plan(i(2), rows)
    assert not calls
    for rows in (1, 8):
        c.plan(i(2), rows)
        assert c.positions.numel() == c.slots.numel() == rows
    assert len(calls) == 2


@pytest.mark.parametrize("present", [False, True])
def test_a_binding_that_is_missing_and_one_that_does_not_load_are_told_apart(present, tmp_path, monkeypatch):
    from bwd_step_b200 import api, build
    if present:
        (tmp_path / "_serving.so").write_bytes(b"no library")
    monkeypatch.setattr(build, "SERVING", str(tmp_path / "_serving.so"))
    monkeypatch.setattr(bwd_step_b200, "__path__", [str(tmp_path)])  # where the package's modules are looked for
    monkeypatch.delattr(bwd_step_b200, "_serving", raising=False)
    monkeypatch.delitem(sys.modules, "bwd_step_b200._serving", raising=False)
    monkeypatch.setattr(api, "_serving_module", None)
    with pytest.raises(RuntimeError, match="does not load.*file too short|does not load.*invalid ELF" if present else "is missing"):
        api._serving()
