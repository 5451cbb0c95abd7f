"""The operators' Python calls refuse tensors of several GPUs, a stream of another one, and sizes
that no tensor has, on the host and before anything is allocated or launched.  The tensors here
have a device, a shape and strides and no memory, so that no GPU is needed."""
import types

import pytest
import torch

from gated_delta_rule_48_gb300 import binding as kb


class Bare(torch.Tensor):
    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError(f"{func} on a tensor without memory")


def bare(shape, dtype=torch.float32, device="cuda:0"):
    return torch.Tensor._make_wrapper_subclass(Bare, shape, dtype=dtype, device=torch.device(device))


E4M3 = torch.float8_e4m3fn
# every tensor that a call takes, by its keyword, with its shape and type
CALLS = {
    "kda_add_rms_norm": dict(x=(4, 256), weight=(256,), residual=(4, 256), y=(4, 256), h=(4, 256)),
    "kda_add_rms_norm_quant": dict(x=(4, 256), weight=(256,), residual=(4, 256),
                                   y=((4, 256), E4M3), y_scale=(4, 2), h=(4, 256)),
    "kda_matmul_fp8": dict(a=((4, 256), E4M3), a_scale=(4, 2), b=((128, 256), E4M3), b_scale=(1, 2),
                           out=(4, 128)),
    "kda_short_conv_fwd": dict(x=(6, 32), weight=(32, 4), bias=(32,), conv_state=(2, 3, 32),
                               cu_seqlens=((3,), torch.int32), y=(6, 32), state_out=(2, 3, 32)),
    "kda_short_conv_step": dict(x=(2, 32), weight=(32, 4), conv_state=(2, 3, 32), bias=(32,),
                                y=(2, 32)),
    "kda_ssm_scan_fwd": dict(x=(6, 32), dt=(6, 32), A=(32, 16), B=(6, 2, 16), C=(6, 2, 16), D=(32,),
                             z=(6, 32), dt_bias=(32,), h0=(2, 32, 16),
                             cu_seqlens=((3,), torch.int32), y=(6, 32), h_final=(2, 32, 16)),
    "kda_ssm_scan_step": dict(x=(2, 32), dt=(2, 32), A=(32, 16), B=(2, 2, 16), C=(2, 2, 16),
                              h=(2, 32, 16), D=(32,), z=(2, 32), dt_bias=(32,), y=(2, 32)),
}


def arguments(name, elsewhere=()):
    made = {}
    for key, what in CALLS[name].items():
        shape, dtype = what if isinstance(what[0], tuple) else (what, torch.float32)
        made[key] = bare(shape, dtype, "cuda:1" if key in elsewhere else "cuda:0")
    return made


@pytest.mark.parametrize("name,key", [(n, k) for n, a in CALLS.items() for k in list(a)[1:]])
def test_an_operand_on_another_gpu_is_refused(name, key):
    with pytest.raises(kb.KdaError, match=f"{key} is on cuda:1, expected cuda:0"):
        getattr(kb, name)(**arguments(name, [key]))


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_gpu_is_refused(name):
    other = types.SimpleNamespace(device=torch.device("cuda:1"))
    with pytest.raises(kb.KdaError, match="the stream is on cuda:1, the tensors on cuda:0"):
        getattr(kb, name)(**arguments(name), stream=other)


@pytest.mark.parametrize("name", ["kda_short_conv_fwd", "kda_ssm_scan_fwd"])
def test_a_negative_number_of_sequences_is_refused(name):
    made = arguments(name)
    made["cu_seqlens"] = made["conv_state" if "conv" in name else "h0"] = None
    made["state_out" if "conv" in name else "h_final"] = None
    with pytest.raises(kb.KdaError, match="n_seqs=-1 is negative"):
        getattr(kb, name)(**made, n_seqs=-1)


@pytest.mark.parametrize("name", ["kda_short_conv_fwd", "kda_short_conv_step"])
def test_a_convolution_of_width_zero_is_refused(name):
    with pytest.raises(kb.KdaError, match="width of 0"):
        getattr(kb, name)(**(arguments(name) | dict(weight=bare((32, 0)))))
