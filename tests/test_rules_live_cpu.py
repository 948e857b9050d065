"""LogitRules hands each call its tensors as they are when the call is made:
pointers, sizes and pitches of resized or replaced storage, never those of its
construction.  The struct is looked at on the host; nothing is launched."""
import pytest
import torch

import entropy_chunked_row_amd as lp

T, V, W = 6, 100, 4


@pytest.fixture
def host_tensors_pass(monkeypatch):
    monkeypatch.setattr(lp, "_same_device", lambda device, named: None)


def _parts():
    return dict(tokens=torch.zeros(T, 9, dtype=torch.int32), hist_len=torch.zeros(T, dtype=torch.int32),
                prompt_len=torch.zeros(T, dtype=torch.int32), row_seq=torch.zeros(T, dtype=torch.int32),
                repetition=torch.ones(T), frequency=torch.ones(T), presence=torch.ones(T),
                bias_offsets=torch.zeros(T + 1, dtype=torch.int64), bias_tokens=torch.zeros(3, dtype=torch.int32),
                bias_values=torch.zeros(3), allowed=torch.zeros(T, W, dtype=torch.int32))


FIELD = dict(row_seq="row_buffer")


def _struct(rules, n=T):
    return rules._check(n, V, torch.device("cpu"))._obj


def _agree(c, d):
    for name, t in d.items():
        assert getattr(c, FIELD.get(name, name)) == t.data_ptr(), name
    assert (c.buffers, c.max_len) == tuple(d["tokens"].shape) and c.ld_tokens == d["tokens"].stride(0)
    assert c.bias_count == d["bias_tokens"].numel() and c.ld_allowed == d["allowed"].stride(0)


def test_replaced_and_resized_tensors(host_tensors_pass):
    d = _parts()
    r = lp.LogitRules(**d)
    _agree(_struct(r), d)
    for name in d:  # another storage
        d[name].data = d[name].clone()
        _agree(_struct(r), d)
    # a larger batch
    n = 64
    for name, t in d.items():
        if name not in ("bias_tokens", "bias_values"):
            t.resize_((n + 1,) if name == "bias_offsets" else (n, *t.shape[1:]))
    d["tokens"].resize_(n, 1000)
    d["bias_tokens"].resize_(500)
    d["bias_values"].resize_(500)
    _agree(_struct(r, n), d)
    # a pitch of its own
    d["allowed"].data = torch.zeros(n, 2 * W, dtype=torch.int32)[:, :W]
    d["tokens"].data = torch.zeros(n, 30, dtype=torch.int32)[:, 5:25]
    _agree(_struct(r, n), d)
    # two calls hold structs of their own
    a, b = _struct(r, n), _struct(r, n)
    a.tokens = 0
    assert b.tokens == d["tokens"].data_ptr()


@pytest.mark.parametrize("name,change,err", [
    ("allowed", lambda t: t.resize_(T, W - 1), ValueError), ("allowed", lambda t: t.resize_(T - 1, W), ValueError),
    ("hist_len", lambda t: t.resize_(T - 1), ValueError), ("row_seq", lambda t: t.resize_(T + 1), ValueError),
    ("bias_offsets", lambda t: t.resize_(T), ValueError), ("bias_values", lambda t: t.resize_(2), ValueError),
    ("tokens", lambda t: t.t_(), ValueError), ("allowed", lambda t: t.transpose_(0, 1), ValueError),
    ("presence", lambda t: setattr(t, "data", torch.ones(2 * T)[::2]), ValueError),
    ("presence", lambda t: setattr(t, "data", torch.ones(T, dtype=torch.float64)), TypeError),
    ("tokens", lambda t: setattr(t, "data", torch.zeros(T, 9, dtype=torch.int64)), TypeError)])
def test_what_no_longer_fits_is_refused(host_tensors_pass, name, change, err):
    d = _parts()
    r = lp.LogitRules(**d)
    _struct(r)
    change(d[name])
    with pytest.raises(err):
        _struct(r)


def test_fewer_buffers_than_rows(host_tensors_pass):
    d = _parts()
    del d["row_seq"]
    r = lp.LogitRules(**d)
    _struct(r)
    d["tokens"].resize_(T - 1, 9)
    with pytest.raises(ValueError, match="buffer"):
        _struct(r)
    d["tokens"].resize_(0, 9)  # nobody has a history
    assert not _struct(r).tokens
