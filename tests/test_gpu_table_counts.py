"""A table whose counts are wrong: more sequences write into a shared page than hold it by its count."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("others", [0, 3])
def test_writers_beyond_the_count_get_nothing(others):
    import adapter_sgmv_bgmv_gb300 as L
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ctx = L.Context(0, max_rows=64)
    # four sequences on page 2, counted twice; `others` on pages of their own
    n = 4 + others
    lens, pages, refs = ints([3] * n), ints([[2, -1]] * 4 + [[3 + i, -1] for i in range(others)]), ints([0, 0, 2] + [1] * others + [0] * 9)
    table = L.PageTable(lens, pages, refs, 4)
    lists = [ints([7] * n) for _ in range(4)]
    was = [t.clone() for t in (lens, pages, refs)]
    L.lora_pages_extend(ctx, table, ints([1] * n), *lists)
    with pytest.raises(L.LoraError) as e:
        ctx.sync_status()
    assert e.value.name == "LORA_E_PAGE"
    assert [v.tolist() for v in lists] == [[0] * 4 + [1] * others, [-1] * n, [-1] * n, [0] * n]
    assert lens.tolist() == [3] * 4 + [4] * others and torch.equal(pages, was[1]) and torch.equal(refs, was[2])
    # as many writers as are counted: the last one keeps the page
    L.lora_pages_extend(ctx, table, ints([0, 2, 0, 2] + [0] * others), *lists)
    ctx.sync_status()
    assert lists[0].tolist() == [0, 2, 0, 2] + [0] * others and lists[1].tolist() == [-1, 2] + [-1] * (n - 2)
    ctx.close()
