"""adjust_logits refuses a status over anything that it reads or writes besides; nothing here touches a GPU."""
from tests.test_cache_abi import P, m  # noqa: F401

R, K, V, WIDTH, N, MASKS = 3, 4, 100, 9, 7, 2
ROWS = R * (1 + K)
NAMES = ("draft", "history", "history_len", "prompt_len", "repetition", "presence", "frequency", "bias_start", "bias_id",
         "bias_value", "mask", "mask_row")
ENTRIES = (R * K, R * WIDTH, R, R, R, R, R, R + 1, N, N, MASKS * 4, ROWS)
AT = {name: 0x100000 + 0x10000 * i for i, name in enumerate(NAMES)}
LOGITS, OUT, STRIDE = 0x400000, 0x500000, 128


def _call(m, status, **other):  # noqa: F811
    at = dict(AT, **other)
    rules = m.SvLogitRules(history_width=WIDTH, bias_entries=N, masks=MASKS, mask_words=4,
                           **{name: at[name] for name in NAMES if name != "draft"})
    rows = [m.SvRows(data, 1, V, STRIDE) for data in (LOGITS, OUT)]
    return m.load().sv_adjust_logits(rows[0], R, K, 1, P(at["draft"]), rules, rows[1], P(status), None)


def test_status_over_inputs(m):  # noqa: F811
    for name, n in zip(NAMES, ENTRIES):
        for status in (AT[name], AT[name] + 4 * (n - 1), AT[name] - 4 * (R - 1)):
            assert _call(m, status) == -1, name
    for data in (LOGITS, OUT):
        for entry in (0, V - 1, -R + 1, STRIDE - R + 1, 3 * STRIDE + 50, (ROWS - 1) * STRIDE + V - 1):
            assert _call(m, data + 4 * entry) == -1, (data, entry)


def test_status_beside_inputs(m):  # noqa: F811
    import torch

    if torch.cuda.is_available():
        return  # these calls are valid
    for name, n in zip(NAMES, ENTRIES):
        assert _call(m, AT[name] + 4 * n) == _call(m, AT[name] - 4 * R) == -8, name
    for data in (LOGITS, OUT):  # ahead of the rows, between them, behind them
        for entry in (-R, V, 5 * STRIDE + V, 5 * STRIDE + STRIDE - R, (ROWS - 1) * STRIDE + V):
            assert _call(m, data + 4 * entry) == -8, (data, entry)
    assert _call(m, AT["mask"] + 40, mask=None, mask_row=None) == -8
